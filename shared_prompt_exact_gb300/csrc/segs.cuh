// segs.cuh -- the response segments of a packed micro-batch as a kernel argument.
//
// The per-token operators (rope.cu, logprobs.cu, policy.cu) need P and R_offsets
// on the device.  The offsets travel in the launch's parameter space (constant
// memory), so a call uploads nothing, keeps nothing and may be captured into a
// graph like any plain launch.  Two capacities are compiled: most micro-batches
// have at most 255 responses and pass 1 KB; up to kMaxSegs pass 16 KB (kernel
// parameters end at 32,764 bytes).
#pragma once
#include <stdint.h>

namespace dkv {

constexpr int kSmallSegs = 255;
constexpr int kMaxSegs = 4095;

template <int CAP>
struct SegTable {
  int32_t P, N;
  int32_t off[CAP + 1];  // off[0..N]
};

// Segment holding response row r (off[0] <= r < off[N]): the largest n with
// off[n] <= r, which is never an empty one.
template <int CAP>
__device__ __forceinline__ int seg_of(const SegTable<CAP>& s, int r) {
  int lo = 0, hi = s.N - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (s.off[mid] <= r) lo = mid;
    else hi = mid - 1;
  }
  return lo;
}

// Position of packed row t: t in the prompt, P + (row within its response) behind it.
template <int CAP>
__device__ __forceinline__ int position_of(const SegTable<CAP>& s, int t) {
  if (t < s.P) return t;
  const int r = t - s.P;
  return s.P + r - s.off[seg_of(s, r)];
}

template <int CAP>
inline SegTable<CAP> make_segs(int P, int N, const int32_t* off) {
  SegTable<CAP> s;
  s.P = P;
  s.N = N;
  for (int n = 0; n <= N; ++n) s.off[n] = off[n];
  return s;
}

}  // namespace dkv
