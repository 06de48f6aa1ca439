// Cutting a cache down to a budget of tokens by accumulated attention weight
// (slot_weights.cu): the choice (dflash_plan_eviction) and the moves that
// follow from it (dflash_move_slots), per (layer, request, kv head).
//
// Of the slots first .. ctx-1 those stay whose token is among the `recent`
// newest, then the heaviest, `budget - first` in all (equal weights: the lower
// slot).  A cache is a set to the attention over it, so no order has to be
// kept: the kept tokens above the budget move into the slots that fall free
// below it, the i-th such token into the i-th such slot, and nothing else
// moves.  A step that drops 16 of 4 112 tokens moves at most 16, where closing
// the gaps would move nearly all.  Sources and targets are disjoint, so the
// moves need no order either.
#include "target.h"
#include "common.cuh"

#include <type_traits>

namespace dflash {
namespace {

// ------------------------------------------------------------------ choice
// The budget-th largest of a list by radix selection over 32-bit keys (11, 11
// and 10 bits), the keys in shared memory: weights and positions are read
// once.  The first digit decides nearly all keys, the few others are set apart:
// compared with each other, or counted by the next two digits.  What stays is a
// bit per slot in a lane's registers, and the moves leave in one piece through
// the keys' place.  Where lists are long or few, a cluster of CTAs shares one:
// each has a stretch of the slots and sends the counts that are not 0 to the
// first, which finds the digit for all.  Bound by instructions and by the
// dependent steps of a list (loads, digits, counts of what moves): 36 layers of
// 8 x 8 lists of 4.1k take 31 us, 11 of them HBM's.  Counts kept two or four
// times over, for lanes that meet in a bin, were slower (45 us against 37), and
// so were weights that came by asynchronous copies (34 against 31).
constexpr int BINS = 2048;
constexpr int FEW = 2048;                     // keys set apart at most
constexpr int MAX_CS = 8;
constexpr uint32_t ZERO = 0x80000000u;        // the key of a weight of 0
constexpr uint32_t PROTECTED = 0xffffffffu;   // the key of a recent token, above every weight's

struct PlanArgs {
  const float *weights;
  const int32_t *positions;
  const int32_t *ctx_len, *seq_len;
  int32_t *moves, *counts, *ctx_out;
  int batch, batch_rows, nkv, capacity;
  int first, recent, budget, top;
  int cs;                      // CTAs per list
  int *status;
};

struct __align__(16) PlanCtrl {
  uint32_t hist[BINS];         // this CTA's counts
  uint32_t warp_sum[32], warp_a[32], warp_b[32];
  uint32_t pick[4];            // the digit of the wanted key, how many keys lie above it, how many have it, and whether those are all 0
  uint32_t ties, holes, movers;   // of this CTA
  uint32_t found, zeros;
  uint32_t few[FEW];           // this CTA's keys that have the first digit of the wanted one
};

// a weight's place in an unsigned order; NaN lies below every number
__device__ __forceinline__ uint32_t weight_key(float v) {
  const uint32_t u = __float_as_uint(v + 0.f);   // -0 and +0 are equal
  return v != v ? 0u : u ^ (static_cast<uint32_t>(static_cast<int32_t>(u) >> 31) | 0x80000000u);
}
__device__ __forceinline__ uint32_t ld_dsmem_u32(uint32_t addr) {
  uint32_t v;
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ void st_dsmem_u32(uint32_t addr, uint32_t v) {
  asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}
__device__ __forceinline__ void add_dsmem_u32(uint32_t addr, uint32_t v) {
  asm volatile("red.relaxed.cluster.shared::cluster.add.u32 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}
// the sum of the first `n` of the warps' values
__device__ __forceinline__ uint32_t sum_before(const uint32_t *v, int n, int lane) {
  return __reduce_add_sync(0xffffffffu, lane < n ? v[lane] : 0u);
}

// T threads; CACHED: a CTA's keys fit its shared memory.
template <int T, bool CACHED>
__global__ void __launch_bounds__(T, T == 256 ? 6 : 1) plan_kernel(const PlanArgs a) {
  constexpr int PLAN_THREADS = T, PLAN_WARPS = T / 32, MINE = BINS / T;   // MINE: bins of a thread
  constexpr int U = T == 256 ? 6 : 8;   // keys of a thread with their loads in flight
  extern __shared__ uint32_t plan_smem[];
  PlanCtrl *ct = reinterpret_cast<PlanCtrl *>(plan_smem);
  uint32_t *keys = plan_smem + sizeof(PlanCtrl) / 4;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int rank = static_cast<int>(blockIdx.x) % a.cs, h = static_cast<int>(blockIdx.x) / a.cs % a.nkv;
  const int lb = static_cast<int>(blockIdx.x) / a.cs / a.nkv, layer = lb / a.batch, b = lb % a.batch;
  auto meet = [&]() {          // the CTAs of the list
    if (a.cs > 1) {
      __syncwarp();
      cluster_sync();
    } else {
      __syncthreads();
    }
  };
  // this thread's bins, the highest first
  const int bin0 = BINS - MINE * (tid + 1);
  using Word = typename std::conditional<MINE % 4 == 0, uint4, uint2>::type;
  constexpr int W = sizeof(Word) / 4;
  static_assert(MINE % W == 0, "bins per thread");
  auto clear = [&] {
#pragma unroll
    for (int i = 0; i < MINE; i += W) *reinterpret_cast<Word *>(&ct->hist[bin0 + i]) = Word();
  };
  clear();
  if (tid == 0) ct->found = ct->zeros = 0;
  // a warp's lanes meet before each half of the barrier: `aligned` wants all of them there
  __syncwarp();
  if (a.cs > 1) asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");   // the counts are cleared
  pdl_start();
  const int ctx = a.ctx_len[b], seq = a.seq_len[b];
  const bool ok = ctx >= 0 && ctx <= a.capacity;
  if (!ok && rank == 0 && h == 0 && layer == 0 && tid == 0) report(a.status, DFLASH_ERR_DEVICE);
  const size_t list = (static_cast<size_t>(layer) * a.batch + b) * a.nkv + h;
  int32_t *into = a.moves + list * 2 * a.top, *source = into + a.top;
  if (rank == 0 && h == 0 && layer == 0 && tid == 0) a.ctx_out[b] = ok ? min(ctx, a.budget) : ctx;
  if (!ok || ctx <= a.budget) {            // nothing to drop
    for (int i = rank * PLAN_THREADS + tid; i < 2 * a.top; i += a.cs * PLAN_THREADS) into[i] = -1;
    if (rank == 0 && tid == 0) a.counts[list] = 0;
    __syncwarp();
    if (a.cs > 1) asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
    return;                                // the whole cluster
  }
  // this CTA's stretch of the slots: whole warps' worths
  const int n = ctx - a.first, per = ((n + a.cs - 1) / a.cs + 31) & ~31;
  const int lo = a.first + min(n, rank * per), mine = min(n, (rank + 1) * per) - min(n, rank * per);
  const size_t row = ((static_cast<size_t>(layer) * a.batch_rows + b) * a.nkv + h) * a.capacity + lo;
  const float *wt = a.weights + row;
  const int32_t *ps = a.positions + row;
  // positions from here on stay
  const int newest = static_cast<int>(max(static_cast<long long>(seq) - a.recent, -0x80000000ll));
  auto make_key = [&](float w, int32_t at) { return at >= newest ? PROTECTED : weight_key(w); };
  auto key_at = [&](int i) { return CACHED ? keys[i] : make_key(wt[i], ps[i]); };
  __syncwarp();
  if (a.cs > 1)                // the counts are cleared
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
  else
    __syncthreads();

  // Each lane looks after 32 neighbouring slots of its warp's stretch (8 or 16 where it
  // is short), GW times, a bit each, and reads its keys in an order that keeps the
  // lanes on banks of their own.  Against 32 slots to a warp, whose masks are ballots
  // and whose moves leave from where they are found, 64 prompts took 70 us for 94.
  constexpr int GW = T == 256 ? 1 : 2;
  const int seg = ((mine + PLAN_WARPS - 1) / PLAN_WARPS + 31) / 32 * 32;   // slots per warp, at most 1024 GW where they are cached
  const int s0 = min(mine, warp * seg), s1 = min(mine, s0 + seg);
  const int log_w = seg <= 256 ? 3 : seg <= 512 ? 4 : 5, width = 1 << log_w;
  auto slot_of = [&](int w) { return s0 + ((32 * w + lane) << log_w); };
  auto mask = [](int n) { return n >= 32 ? 0xffffffffu : n <= 0 ? 0u : (1u << n) - 1; };   // the lowest n bits
  uint32_t up[GW], eq[GW];     // slots whose key's bits from `shift` on lie above `value`, and those that equal it
  auto look = [&](int shift, uint32_t value) {
#pragma unroll
    for (int w = 0; w < GW; ++w) {
      const int g = slot_of(w);
      up[w] = eq[w] = 0;
      if (g >= s1) continue;
#pragma unroll 8
      for (int j = 0; j < width; ++j) {
        const int r = (j + (lane >> (5 - log_w))) & (width - 1);
        const uint32_t k = keys[g + r] >> shift;
        if (k > value) up[w] |= 1u << r;
        if (k == value) eq[w] |= 1u << r;
      }
      up[w] &= mask(s1 - g);
      eq[w] &= mask(s1 - g);
    }
  };
  auto scan = [&](uint32_t v) {   // of the lanes up to this one
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t t = __shfl_up_sync(0xffffffffu, v, o);
      if (lane >= o) v += t;
    }
    return v;
  };

  // ---- radix selection: `want` keys are to stay, those with the found prefix above them already
  uint32_t want = a.budget - a.first, prefix = 0, ties_all = 0;
  int n_few = -1;              // keys with the first digit, where they were few enough to be set apart
#pragma unroll
  for (int pass = 0; pass < 3; ++pass) {
    const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0, bits = pass == 2 ? 10 : 11, above = shift + bits;
    uint32_t zeros = 0, prot = 0;          // the two keys that many slots may share, counted without atomics
    auto count = [&](uint32_t k, bool in) {
      if (pass > 0) in = in && (k >> (above & 31)) == prefix;
      zeros += in && k == ZERO;
      prot += in && k == PROTECTED;
      if (in && k != ZERO && k != PROTECTED) atomicAdd(&ct->hist[(k >> shift) & ((1u << bits) - 1)], 1u);
    };
    if (pass > 0 && n_few >= 0) {
      for (int i = tid; i < n_few; i += PLAN_THREADS) count(ct->few[i], true);
    } else if (pass > 0 && CACHED) {
#pragma unroll 4
      for (int i = tid; i < mine; i += PLAN_THREADS) count(keys[i], true);
    } else {
      // (the last ones with the others in one batch: a loop of their own is a latency of its own)
      for (int i = tid; i < mine; i += U * PLAN_THREADS) {
        float w[U];
        int32_t at[U];
#pragma unroll
        for (int u = 0; u < U; ++u)
          if (i + u * PLAN_THREADS < mine) {
            w[u] = wt[i + u * PLAN_THREADS];
            at[u] = ps[i + u * PLAN_THREADS];
          }
#pragma unroll
        for (int u = 0; u < U; ++u)
          if (i + u * PLAN_THREADS < mine) {
            const uint32_t k = make_key(w[u], at[u]);
            if (CACHED) keys[i + u * PLAN_THREADS] = k;
            count(k, true);
          }
      }
    }
    zeros = __reduce_add_sync(0xffffffffu, zeros);
    prot = __reduce_add_sync(0xffffffffu, prot);
    if (lane == 0) {
      if (zeros && pass == 0) {
        if (a.cs > 1)
          add_dsmem_u32(dsmem_addr(&ct->zeros, 0), zeros);
        else
          atomicAdd(&ct->zeros, zeros);
      }
      if (zeros) atomicAdd(&ct->hist[(ZERO >> shift) & ((1u << bits) - 1)], zeros);
      if (prot) atomicAdd(&ct->hist[(PROTECTED >> shift) & ((1u << bits) - 1)], prot);
    }
    uint32_t c[MINE], sum = 0;
    auto take = [&] {          // this thread's counts, cleared for the next pass
#pragma unroll
      for (int i = 0; i < MINE; i += W) {
        *reinterpret_cast<Word *>(&c[i]) = *reinterpret_cast<const Word *>(&ct->hist[bin0 + i]);
        *reinterpret_cast<Word *>(&ct->hist[bin0 + i]) = Word();
      }
    };
    if (a.cs > 1) {
      if (rank > 0) {
        __syncthreads();
        take();
#pragma unroll
        for (int i = 0; i < MINE; ++i)
          if (c[i]) add_dsmem_u32(dsmem_addr(&ct->hist[bin0 + i], 0), c[i]);
      }
      meet();
    } else {
      __syncthreads();
    }
    if (rank == 0) {           // the bin that holds the want-th largest key
      take();
#pragma unroll
      for (int i = 0; i < MINE; ++i) sum += c[i];
      uint32_t inc = sum;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const uint32_t t = __shfl_up_sync(0xffffffffu, inc, o);
        if (lane >= o) inc += t;
      }
      if (lane == 31) ct->warp_sum[warp] = inc;
      __syncthreads();
      uint32_t over = sum_before(ct->warp_sum, warp, lane) + inc - sum;   // keys above this thread's bins
      if (over < want && want <= over + sum) {
        int bin = bin0;        // this thread's, from the top down
        uint32_t has = 0;
#pragma unroll
        for (int u = MINE - 1; u >= 0; --u)
          if (has == 0) {
            if (want <= over + c[u])
              has = c[u], bin = bin0 + u;
            else
              over += c[u];
          }
        const uint32_t all_zero = pass == 0 && bin == static_cast<int>(ZERO >> 21) && has == ct->zeros;
        if (a.cs == 1) {
          ct->pick[0] = bin, ct->pick[1] = over, ct->pick[2] = has, ct->pick[3] = all_zero;
        } else {
          for (int r = 0; r < a.cs; ++r) {
            const uint32_t to = dsmem_addr(ct->pick, r);
            st_dsmem_u32(to, bin);
            st_dsmem_u32(to + 4, over);
            st_dsmem_u32(to + 8, has);
            st_dsmem_u32(to + 12, all_zero);
          }
        }
      }
    }
    meet();
    prefix = pass == 0 ? ct->pick[0] : (prefix << bits) | ct->pick[0];
    want -= ct->pick[1];
    ties_all = ct->pick[2];
    // Tokens that nobody attended to may be many: their key needs no more digits (36
    // layers, a third of the weights 0: 31 us, 50 with them).
    if (pass == 0 && ct->pick[3]) {
      prefix = ZERO;
      break;
    }
    if (pass == 0 && CACHED) {
      look(21, prefix);
      uint32_t have = 0;
#pragma unroll
      for (int w = 0; w < GW; ++w) have += __popc(eq[w]);
      const uint32_t inc = scan(have);
      uint32_t at = 0;
      if (lane == 31 && inc) at = atomicAdd(&ct->found, inc);
      at = __shfl_sync(0xffffffffu, at, 31) + inc - have;
#pragma unroll
      for (int w = 0; w < GW; ++w)
        for (uint32_t e = eq[w]; e && at < FEW; e &= e - 1, ++at) ct->few[at] = keys[slot_of(w) + __ffs(e) - 1];
      __syncthreads();
      if (ct->found <= FEW) n_few = static_cast<int>(ct->found);
      if (a.cs == 1 && n_few >= 0 && n_few <= 256) {
        // each compared with all of them, by the warps that hold one; with the loads above in
        // one batch the 36 layers took 38 us for 45. All 1024 threads against as many
        // candidates took 171 us for 101 on 64 prompts
        const bool holds = (tid & ~31) < n_few;
        const uint32_t k = tid < n_few ? ct->few[tid] : 0u;
        uint32_t more = 0, same = 0;
#pragma unroll 4
        for (int i = 0; i < (holds ? n_few : 0); ++i) {
          const uint32_t x = ct->few[i];
          more += x > k;
          same += x == k;
        }
        __syncthreads();       // everybody has read what the first digit's pick says
        if (tid < n_few && more < want && want <= more + same) {   // equal keys write the same
          ct->pick[0] = k;
          ct->pick[1] = more;
          ct->pick[2] = same;
        }
        __syncthreads();
        prefix = ct->pick[0];
        want -= ct->pick[1];
        ties_all = ct->pick[2];
        break;
      }
    }
  }
  // keys above `prefix` stay, and `want` of the ties_all that equal it: the lowest slots
  uint32_t tie_base = 0;       // equal keys in slots before this warp's
  auto count_ties = [&](uint32_t t) {   // t: this warp's
    if (lane == 0) ct->warp_a[warp] = t;
    __syncthreads();
    tie_base = sum_before(ct->warp_a, warp, lane);
    if (a.cs > 1) {
      const uint32_t all = sum_before(ct->warp_a, PLAN_WARPS, lane);
      if (tid == 0) ct->ties = all;
      meet();
      for (int r = 0; r < rank; ++r) tie_base += ld_dsmem_u32(dsmem_addr(&ct->ties, r));
    }
    __syncthreads();
  };
  const int keep = a.budget;   // ctx > budget here
  auto under = [&](int i0) { return mask(keep - lo - i0); };   // of 32 slots from i0 on, those below `keep`
  uint32_t hole0 = 0, mover0 = 0, count = 0;   // of the CTAs before this one; in all: as many holes as movers
  auto count_moves = [&](uint32_t holes, uint32_t movers) {    // this warp's
    if (lane == 0) {
      ct->warp_a[warp] = holes;
      ct->warp_b[warp] = movers;
    }
    __syncthreads();
    count = sum_before(ct->warp_a, PLAN_WARPS, lane);
    if (a.cs > 1) {
      const uint32_t y = sum_before(ct->warp_b, PLAN_WARPS, lane);
      if (tid == 0) {
        ct->holes = count;
        ct->movers = y;
      }
      meet();
      count = 0;
      for (int r = 0; r < a.cs; ++r) {
        const uint32_t x = ld_dsmem_u32(dsmem_addr(&ct->holes, r));
        count += x;
        if (r < rank) {
          hole0 += x;
          mover0 += ld_dsmem_u32(dsmem_addr(&ct->movers, r));
        }
      }
    }
    __syncwarp();
  };
  if constexpr (CACHED) {
    uint32_t tie[GW];
    if (n_few >= 0) {          // what the first digit left open
#pragma unroll
      for (int w = 0; w < GW; ++w) {
        tie[w] = 0;
        for (uint32_t e = eq[w]; e; e &= e - 1) {
          const uint32_t k = keys[slot_of(w) + __ffs(e) - 1], bit = e & (0u - e);
          if (k > prefix) up[w] |= bit;
          if (k == prefix) tie[w] |= bit;
        }
      }
    } else {
      look(0, prefix);
#pragma unroll
      for (int w = 0; w < GW; ++w) tie[w] = eq[w];
    }
    if (want < ties_all) {
      uint32_t t = 0;
#pragma unroll
      for (int w = 0; w < GW; ++w) t += __popc(tie[w]);
      count_ties(__reduce_add_sync(0xffffffffu, t));
#pragma unroll
      for (int w = 0; w < GW; ++w) {
        const uint32_t n = __popc(tie[w]), inc = scan(n), before = tie_base + inc - n;
        const uint32_t some = before < want ? want - before : 0;
        if (some < n) {        // the lowest of them
          uint32_t rest = tie[w];
          for (uint32_t i = 0; i < some; ++i) rest &= rest - 1;
          tie[w] ^= rest;
        }
        tie_base += __shfl_sync(0xffffffffu, inc, 31);
      }
    }
    // what falls free below `keep` and what is kept from it on; both counts in one sum
    uint32_t hole[GW], mover[GW], off[GW], sum = 0;
#pragma unroll
    for (int w = 0; w < GW; ++w) {
      const uint32_t in = mask(min(width, s1 - slot_of(w))), low = under(slot_of(w)), stays = up[w] | tie[w];
      hole[w] = ~stays & low & in;
      mover[w] = stays & ~low & in;
      const uint32_t n = __popc(hole[w]) | __popc(mover[w]) << 16, inc = scan(n);
      off[w] = sum + inc - n;
      sum += __shfl_sync(0xffffffffu, inc, 31);
    }
    count_moves(sum & 0xffffu, sum >> 16);
    // the slots in their order, in the keys' place, which everybody has read
    const uint32_t holes = sum_before(ct->warp_a, PLAN_WARPS, lane), movers = sum_before(ct->warp_b, PLAN_WARPS, lane);
    const uint32_t h0 = sum_before(ct->warp_a, warp, lane), m0 = holes + sum_before(ct->warp_b, warp, lane);
#pragma unroll
    for (int w = 0; w < GW; ++w) {
      uint32_t *to = keys + h0 + (off[w] & 0xffffu);
      for (uint32_t e = hole[w]; e; e &= e - 1) *to++ = lo + slot_of(w) + __ffs(e) - 1;
      to = keys + m0 + (off[w] >> 16);
      for (uint32_t e = mover[w]; e; e &= e - 1) *to++ = lo + slot_of(w) + __ffs(e) - 1;
    }
    __syncthreads();
#pragma unroll 4
    for (uint32_t i = tid; i < holes; i += PLAN_THREADS) into[hole0 + i] = keys[i];
#pragma unroll 4
    for (uint32_t i = tid; i < movers; i += PLAN_THREADS) source[mover0 + i] = keys[holes + i];
  } else {
    if (want < ties_all) {
      uint32_t t = 0;
      for (int i0 = s0; i0 < s1; i0 += 32)
        t += __popc(__ballot_sync(0xffffffffu, i0 + lane < s1 && key_at(i0 + lane) == prefix));
      count_ties(t);
    }
    const uint32_t below = (1u << lane) - 1;
    // Of 32 slots from i0 on, those that fall free below `keep` and those kept from
    // it on, a bit each; `tie` counts the equal keys before.
    auto flags = [&](int i0, uint32_t &tie) {
      const int i = i0 + lane;
      const bool in = i < s1;
      const uint32_t k = in ? key_at(i) : 0u;
      bool stays = k >= prefix;
      if (want < ties_all) {
        const uint32_t eq = __ballot_sync(0xffffffffu, in && k == prefix);
        stays = k > prefix || (k == prefix && tie + __popc(eq & below) < want);
        tie += __popc(eq);
      }
      return __ballot_sync(0xffffffffu, in && stays == (lo + i >= keep));
    };
    uint32_t holes = 0, movers = 0, tie = tie_base;
    for (int i0 = s0; i0 < s1; i0 += 32) {
      const uint32_t f = flags(i0, tie), u = under(i0);
      holes += __popc(f & u);
      movers += __popc(f & ~u);
    }
    count_moves(holes, movers);
    uint32_t hole = hole0 + sum_before(ct->warp_a, warp, lane), mover = mover0 + sum_before(ct->warp_b, warp, lane);
    tie = tie_base;
    for (int i0 = s0; i0 < s1; i0 += 32) {
      const uint32_t f = flags(i0, tie), u = under(i0);
      if (f >> lane & 1) {
        if (u >> lane & 1)
          into[hole + __popc(f & u & below)] = lo + i0 + lane;
        else
          source[mover + __popc(f & ~u & below)] = lo + i0 + lane;
      }
      hole += __popc(f & u);
      mover += __popc(f & ~u);
    }
  }
  for (int i = static_cast<int>(count) + rank * PLAN_THREADS + tid; i < a.top; i += a.cs * PLAN_THREADS)
    into[i] = source[i] = -1;
  if (rank == 0 && tid == 0) a.counts[list] = static_cast<int32_t>(count);
  if (a.cs > 1) {
    __syncwarp();
    cluster_sync();            // no CTA leaves while its counts are read
  }
}

// ------------------------------------------------------------------ moves
// A CTA takes 32 moves of a list.  K rows are copied 16 bytes a lane; V lies
// transposed, so a lane is a move and the warps walk the dims: targets and
// sources ascend, and neighbouring lanes share the sectors of a page's row
// where they are dense.  Bound by the sectors touched, 32 bytes for a value
// where the moves are sparse, and with few moves by the way to them (count and
// moves, then pages, then the values): the loads of K and V are all in flight
// before the first store.
constexpr int MOVE_THREADS = 256, PER_CTA = 32;

struct MoveArgs {
  void *k, *v;                 // the first layer's
  long long layer_elems;
  float *weights;
  int32_t *positions;
  const int32_t *moves, *counts, *page_table;
  int batch, batch_rows, nkv, capacity, top;
  int max_pages, num_pages;
  int *status;
};

template <typename V, int D>   // V: an unsigned integer as wide as the values
__global__ void __launch_bounds__(MOVE_THREADS) move_kernel(const MoveArgs a) {
  constexpr int VEC = 16 / sizeof(V), LPR = D / VEC, STEP = MOVE_THREADS / 32;
  __shared__ long long s_to[PER_CTA], s_of[PER_CTA];   // (page x kv heads + head) x 64 + slot, -1: no move
  __shared__ int2 s_slot[PER_CTA];                     // the request's slots
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int list = blockIdx.x, h = list % a.nkv, b = list / a.nkv % a.batch, layer = list / a.nkv / a.batch;
  pdl_start();
  V *v = static_cast<V *>(a.v) + layer * a.layer_elems;
  uint4 *k = reinterpret_cast<uint4 *>(static_cast<V *>(a.k) + layer * a.layer_elems);
  const int32_t *moves = a.moves + static_cast<size_t>(list) * 2 * a.top;
  const size_t row = ((static_cast<size_t>(layer) * a.batch_rows + b) * a.nkv + h) * a.capacity;
  for (int i0 = blockIdx.y * PER_CTA; i0 < a.top; i0 += gridDim.y * PER_CTA) {
    const int count = a.counts[list];
    if (count < 0 || count > a.top) {
      if (blockIdx.y == 0 && tid == 0) report(a.status, DFLASH_ERR_DEVICE);
      return;
    }
    if (i0 >= count) return;
    if (warp == 0) {
      long long to = -1, of = -1;
      int into = 0, source = 0;
      if (i0 + lane < a.top) {   // whether it counts or not: the loads need not wait for the count
        into = moves[i0 + lane];
        source = moves[a.top + i0 + lane];
      }
      if (i0 + lane < count) {
        const int most = min(a.capacity, a.max_pages * PAGE);
        bool ok = into >= 0 && into < most && source >= 0 && source < most;
        if (ok) {
          const int32_t *table = a.page_table + static_cast<size_t>(b) * a.max_pages;
          const int p0 = table[into / PAGE], p1 = table[source / PAGE];
          ok = p0 >= 0 && p0 < a.num_pages && p1 >= 0 && p1 < a.num_pages;
          if (ok) {
            to = (static_cast<long long>(p0) * a.nkv + h) * PAGE + into % PAGE;
            of = (static_cast<long long>(p1) * a.nkv + h) * PAGE + source % PAGE;
          }
        }
        if (!ok) report(a.status, DFLASH_ERR_DEVICE);
      }
      s_to[lane] = to;
      s_of[lane] = of;
      s_slot[lane] = make_int2(into, source);
    }
    __syncthreads();
    // K [page][head][slot][d]
    constexpr int KN = PER_CTA * LPR / MOVE_THREADS;
    uint4 kx[KN];
#pragma unroll
    for (int u = 0; u < KN; ++u) {
      const int e = u * MOVE_THREADS + tid, i = e / LPR, c = e % LPR;
      if (s_to[i] >= 0) kx[u] = k[s_of[i] * LPR + c];
    }
    // V [page][head][d][slot]: lane = move
    const long long to = s_to[lane], of = s_of[lane];
    const V *src = v + (of / PAGE) * (D * PAGE) + of % PAGE;
    V *dst = v + (to / PAGE) * (D * PAGE) + to % PAGE;
    V x[D / STEP];
    float wt = 0.f;
    int32_t at = 0;
    if (to >= 0) {
#pragma unroll
      for (int u = 0; u < D / STEP; ++u) x[u] = src[(u * STEP + warp) * PAGE];
      if (warp == 0) {
        wt = a.weights[row + s_slot[lane].y];
        at = a.positions[row + s_slot[lane].y];
      }
    }
#pragma unroll
    for (int u = 0; u < KN; ++u) {
      const int e = u * MOVE_THREADS + tid, i = e / LPR, c = e % LPR;
      if (s_to[i] >= 0) k[s_to[i] * LPR + c] = kx[u];
    }
    if (to >= 0) {
#pragma unroll
      for (int u = 0; u < D / STEP; ++u) dst[(u * STEP + warp) * PAGE] = x[u];
      if (warp == 0) {
        a.weights[row + s_slot[lane].x] = wt;
        a.positions[row + s_slot[lane].x] = at;
      }
    }
    __syncthreads();
  }
}

}  // namespace
}  // namespace dflash

using namespace dflash;

extern "C" {

DFLASH_API int dflash_plan_eviction(const dflash_heads *hs, const dflash_slots *slots, int layer, int n_layers,
                                    const int32_t *ctx_len, const int32_t *seq_len, int batch, int first, int recent,
                                    int budget, int32_t *moves, int top, int32_t *counts, int32_t *ctx_out,
                                    void *workspace, size_t workspace_bytes, dflash_stream_t stream) {
  const char *who = "plan_eviction";
  if (int e = check_heads(who, hs)) return e;
  if (int e = check_slots(who, slots, batch)) return e;
  if (!workspace || (batch > 0 && (!ctx_len || !seq_len || !ctx_out))) return set_error(DFLASH_ERR_ARG, "%s: null argument", who);
  if (batch < 0 || layer < 0 || n_layers < 0 || first < 0 || recent < 0 || budget < 1 || budget > (1 << 24) ||
      static_cast<long long>(first) + recent > budget || first >= budget)
    return set_error(DFLASH_ERR_ARG, "%s: batch, layers, first, recent or budget out of range (first < budget, first + recent <= budget)", who);
  if (top > (1 << 24))   // no list has as many slots
    return set_error(DFLASH_ERR_ARG, "%s: top must be at most 2^24", who);
  const int room = budget - first, over = slots->capacity - budget, most = room < over ? room : over > 0 ? over : 0;
  if (top < most) return set_error(DFLASH_ERR_SHAPE, "%s: room for %d moves, %d needed", who, top, most);
  if (batch > 0 && n_layers > 0 && (!counts || (top > 0 && !moves))) return set_error(DFLASH_ERR_ARG, "%s: null argument", who);
  if (off_words(ctx_len, seq_len, moves, counts, ctx_out) || (reinterpret_cast<uintptr_t>(workspace) & 15))
    return set_error(DFLASH_ERR_ALIGN, "%s: arrays must be aligned to their elements, the workspace to 16 bytes", who);
  if (workspace_bytes < 256) return set_error(DFLASH_ERR_SHAPE, "%s: workspace of %zu bytes, 256 needed", who, workspace_bytes);
  if (batch == 0 || n_layers == 0) return DFLASH_OK;
  const long long lists = static_cast<long long>(n_layers) * batch * hs->n_kv_heads;
  if (lists > (1 << 27)) return set_error(DFLASH_ERR_SHAPE, "%s: too many layers x requests x kv heads", who);
  // one CTA writes a request's length while those of other lists may not have read it yet
  auto over_it = [&](const int32_t *in) {
    const uintptr_t x = reinterpret_cast<uintptr_t>(in), y = reinterpret_cast<uintptr_t>(ctx_out);
    return (x < y ? y - x : x - y) < batch * sizeof(int32_t);
  };
  if (over_it(ctx_len) || over_it(seq_len)) return set_error(DFLASH_ERR_ARG, "%s: ctx_out lies over ctx_len or seq_len", who);
  Device dev;
  if (int e = current_device(&dev)) return e;
  const size_t at = static_cast<size_t>(layer) * slots->batch_rows * hs->n_kv_heads * slots->capacity;
  PlanArgs a = {};
  a.weights = slots->weights + at;
  a.positions = slots->positions + at;
  a.ctx_len = ctx_len;
  a.seq_len = seq_len;
  a.moves = moves;
  a.counts = counts;
  a.ctx_out = ctx_out;
  a.batch = batch;
  a.batch_rows = slots->batch_rows;
  a.nkv = hs->n_kv_heads;
  a.capacity = slots->capacity;
  a.first = first;
  a.recent = recent;
  a.budget = budget;
  a.top = top;
  a.status = static_cast<int *>(workspace);
  // A CTA per list as long as its keys fit, 256 threads up to 8192 slots and 1024
  // beyond (64 x 8 lists of 16k..32k slots 69 us; on clusters of two, whose meetings
  // cost more than the emptier SM, 139 when it was 101); where lists are few, a
  // cluster (8 lists of 131071: 19 us on eight CTAs each).
  a.cs = 1;
  const int short_list = 8192, longest = 49152;
  while (a.cs < MAX_CS && (slots->capacity / a.cs > longest || (lists * a.cs * 2 <= dev.sms && slots->capacity / a.cs > 4096)))
    a.cs *= 2;
  const int per = ((slots->capacity + a.cs - 1) / a.cs + 31) & ~31, limit = 227 << 10;
  const bool cached = static_cast<int>(sizeof(PlanCtrl)) + per * 4LL <= limit;
  const int smem = static_cast<int>(sizeof(PlanCtrl)) + (cached ? per * 4 : 0);
  const bool wide = per > short_list;
  static std::atomic<uint64_t> smem_set[3];
  auto *kernel = !cached ? plan_kernel<1024, false> : wide ? plan_kernel<1024, true> : plan_kernel<256, true>;
  const int which = !cached ? 0 : wide ? 1 : 2;
  if (int e = allow_smem(smem_set[which], dev, kernel, limit)) return e;
  // as many CTAs on an SM as its shared memory holds, not a default split with L1
  static std::atomic<uint64_t> carved[3];
  const uint64_t bit = dev.index < 64 ? 1ull << dev.index : 0;
  if (!(carved[which].load(std::memory_order_relaxed) & bit)) {
    if (int e = cuda_check(cudaFuncSetAttribute(kernel, cudaFuncAttributePreferredSharedMemoryCarveout, cudaSharedmemCarveoutMaxShared),
                           "shared memory carveout"))
      return e;
    carved[which].fetch_or(bit, std::memory_order_relaxed);
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(lists * a.cs));
  cfg.blockDim = dim3(cached && !wide ? 256 : 1024);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = reinterpret_cast<cudaStream_t>(stream);
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = a.cs;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = a.cs > 1 ? 2 : 1;
  return cuda_check(cudaLaunchKernelEx(&cfg, kernel, a), "plan_eviction launch");
}

DFLASH_API int dflash_move_slots(const dflash_heads *hs, const dflash_kv *kv, const dflash_slots *slots, int layer,
                                 int n_layers, const int32_t *moves, int top, const int32_t *counts, int batch,
                                 void *workspace, size_t workspace_bytes, dflash_stream_t stream) {
  const char *who = "move_slots";
  if (int e = check_heads(who, hs)) return e;
  static const int32_t none[2] = {0, 0};   // no rows, no requests: the cache's own checks are what is wanted
  if (int e = check_target(who, hs, kv, layer, nullptr, 8, 8, none, 0, none, batch, workspace, workspace_bytes, 256)) return e;
  if (int e = check_slots(who, slots, batch)) return e;
  if (n_layers < 0 || top < 0 || top > (1 << 24)) return set_error(DFLASH_ERR_ARG, "%s: n_layers or top out of range", who);
  if (batch > 0 && n_layers > 0 && top > 0 && (!moves || !counts)) return set_error(DFLASH_ERR_ARG, "%s: null argument", who);
  if (off_words(moves, counts)) return set_error(DFLASH_ERR_ALIGN, "%s: moves and counts must be aligned to their elements", who);
  const long long lists = static_cast<long long>(n_layers) * batch * hs->n_kv_heads;
  if (lists > (1 << 27)) return set_error(DFLASH_ERR_SHAPE, "%s: too many layers x requests x kv heads", who);
  if (batch == 0 || n_layers == 0 || top == 0) return DFLASH_OK;
  const size_t off = layer_offset(*hs, *kv, layer) * elt_bytes(*hs);
  const size_t at = static_cast<size_t>(layer) * slots->batch_rows * hs->n_kv_heads * slots->capacity;
  MoveArgs a = {};
  a.k = static_cast<char *>(kv->k_cache) + off;
  a.v = static_cast<char *>(kv->v_cache) + off;
  a.layer_elems = static_cast<long long>(layer_offset(*hs, *kv, 1));
  a.weights = slots->weights + at;
  a.positions = slots->positions + at;
  a.moves = moves;
  a.counts = counts;
  a.page_table = kv->page_table;
  a.batch = batch;
  a.batch_rows = slots->batch_rows;
  a.nkv = hs->n_kv_heads;
  a.capacity = slots->capacity;
  a.top = top;
  a.max_pages = kv->max_pages;
  a.num_pages = kv->num_pages;
  a.status = static_cast<int *>(workspace);
  const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  auto kernel = hs->dtype == DFLASH_F32 ? (hs->head_dim == 64 ? move_kernel<uint32_t, 64> : move_kernel<uint32_t, 128>)
                                        : (hs->head_dim == 64 ? move_kernel<uint16_t, 64> : move_kernel<uint16_t, 128>);
  const int parts = (top + PER_CTA - 1) / PER_CTA;
  const dim3 grid(static_cast<unsigned>(lists), static_cast<unsigned>(parts < 4096 ? parts : 4096));
  return cuda_check(launch_pdl(kernel, grid, dim3(MOVE_THREADS), 0, s, a), "move_slots launch");
}

}  // extern "C"
