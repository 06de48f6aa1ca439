// Rotary position angles shared by the row kernels and the cache append:
// theta_i = base^(-2i/d) tabulated on the host in fp64 as fp32 (hi, lo)
// pairs, cos / sin of pos * theta_i formed in fp32 on the device.
#pragma once

#include <math.h>

namespace dflash {

// cos / sin of pos * theta_i, theta_i = hi + lo (host-computed in fp64), all
// in fp32 (this GPU's fp64 rate is a small fraction of fp32's): the product
// pos * hi is split exactly into prod + err by one FMA, whole turns are
// removed from prod with 2 pi in three parts (Cody-Waite: 6.28125 has few
// significant bits; the rest in two fp32 terms), and the small terms are
// added back.  The angle's error is three roundings of values below 4 up to
// position 2^22: below 4e-7 rad (3.6e-7 found).  Up to 2^24 the turns of prod
// are off by up to 1/6 and tail reaches 1, so that r and r + tail pass 4:
// below 8.5e-7 (7.1e-7 found).
__device__ __forceinline__ void rope_cs(int pos, float th_hi, float th_lo, float &c, float &s) {
  const float p = static_cast<float>(pos);        // exact below 2^24
  const float prod = p * th_hi;
  const float err = fmaf(p, th_hi, -prod);        // p * th_hi = prod + err exactly
  const float tail = fmaf(p, th_lo, err);
  const float k = rintf(prod * 0.15915494309189535f);   // whole turns
  float r = fmaf(-k, 6.28125f, prod);
  r = fmaf(-k, 1.9353072e-3f, r);
  r = fmaf(-k, 1.0253132e-11f, r);
  sincosf(r + tail, &s, &c);
}

struct RopeArgs {
  float th_hi[64], th_lo[64];
};

// This lane's angles theta_{lane + 32 i}, i < N, from the parameter table.
// Kernel parameters indexed by lane serialise the constant bank (one access
// per distinct address, each a possible miss); uniform reads broadcast, so
// the warp walks the table uniformly and each lane keeps its entries.
template <int N>
__device__ __forceinline__ void lane_thetas(const RopeArgs &rp, int lane, float (&hi)[N], float (&lo)[N]) {
#pragma unroll
  for (int i = 0; i < N; ++i) hi[i] = lo[i] = 0.f;
#pragma unroll 4
  for (int k = 0; k < 32; ++k) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const float h = rp.th_hi[k + 32 * i], l = rp.th_lo[k + 32 * i];
      if (lane == k) {
        hi[i] = h;
        lo[i] = l;
      }
    }
  }
}

inline RopeArgs rope_table(int d, float base) {
  RopeArgs r = {};
  for (int i = 0; i < d / 2 && i < 64; ++i) {
    const double th = pow(static_cast<double>(base), -2.0 * i / d);
    r.th_hi[i] = static_cast<float>(th);
    r.th_lo[i] = static_cast<float>(th - static_cast<double>(r.th_hi[i]));
  }
  return r;
}

}  // namespace dflash
