// twofloat.cuh -- numbers as the unevaluated sum of two floats (some 46 bits), by error-free sums and products (Dekker;
// Knuth).  A dependent operation takes 4 cycles where one in fp64 takes tens.
#pragma once
#include <stdint.h>

namespace dkv {

namespace {

struct Two {
  float hi, lo;
};

// products on their own: never contracted with the sum that takes them
__host__ __device__ __forceinline__ float product(float a, float b) {
#ifdef __CUDA_ARCH__
  return __fmul_rn(a, b);
#else
  return a * b;
#endif
}
__host__ __device__ __forceinline__ Two two_sum(float a, float b) {
  const float s = a + b, t = s - a;
  return Two{s, (a - (s - t)) + (b - t)};
}
__host__ __device__ __forceinline__ Two fast_sum(float a, float b) {  // |a| >= |b|
  const float s = a + b;
  return Two{s, b - (s - a)};
}
__host__ __device__ __forceinline__ Two two_product(float a, float b) {
  const float p = product(a, b);
  return Two{p, fmaf(a, b, -p)};
}
// Off by 2^-46 of |a| + |b|, of |a b|.
__host__ __device__ __forceinline__ Two operator+(Two a, Two b) {
  const Two s = two_sum(a.hi, b.hi);
  return fast_sum(s.hi, s.lo + (a.lo + b.lo));
}
__host__ __device__ __forceinline__ Two operator*(Two a, Two b) {
  const Two p = two_product(a.hi, b.hi);
  return fast_sum(p.hi, fmaf(a.hi, b.lo, fmaf(a.lo, b.hi, p.lo)));
}
__host__ __device__ __forceinline__ Two operator-(Two a) { return Two{-a.hi, -a.lo}; }
__host__ __device__ constexpr Two two(double x) { return Two{(float)x, (float)(x - (double)(float)x)}; }

// Cosine and sine of `turns` 2^-64 turns, off by 2^-44: the nearest quarter off, Taylor's series of what is left (up to
// pi / 4).
__host__ __device__ __forceinline__ void cos_sin_turns(uint64_t turns, Two& c, Two& s) {
  const uint32_t quarter = (uint32_t)((turns + (1ull << 61)) >> 62);  // 4 of them is 0 again
  const int64_t rest = (int64_t)(turns - ((uint64_t)quarter << 62));
  const float hi = (float)rest;
  const Two x = Two{hi * 0x1p-63f, (float)(rest - (int64_t)hi) * 0x1p-63f} * two(3.14159265358979323846), z = x * x;
  const float z1 = z.hi;
  const float s9 = fmaf(fmaf(fmaf((float)(-1 / 1307674368000.0), z1, (float)(1 / 6227020800.0)), z1, (float)(-1 / 39916800.0)), z1,
                        (float)(1 / 362880.0));
  const float c10 = fmaf(fmaf(fmaf((float)(1 / 20922789888000.0), z1, (float)(-1 / 87178291200.0)), z1, (float)(1 / 479001600.0)), z1,
                         (float)(-1 / 3628800.0));
  const Two one{1.f, 0.f};
  Two sn = two(-1 / 5040.0) + two_product(z1, s9), cs = two(1 / 40320.0) + two_product(z1, c10);
  sn = x * (one + z * (two(-1 / 6.0) + z * (two(1 / 120.0) + z * sn)));
  cs = one + z * (two(-0.5) + z * (two(1 / 24.0) + z * (two(-1 / 720.0) + z * cs)));
  const bool swap = quarter & 1;
  c = swap ? sn : cs;
  s = swap ? cs : sn;
  if ((quarter + 1) & 2) c = -c;
  if (quarter & 2) s = -s;
}

}  // namespace

}  // namespace dkv
