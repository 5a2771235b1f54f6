// rope.cuh -- a head's values over the lanes of a warp: the two 16-byte vectors that each of
// D / 16 lanes holds, the position rotation of a row and the loads that run ahead through
// shared memory.  Used by rope.cu (packed rows) and cache.cu (rows that enter the cache).
#pragma once
#include <cuda_bf16.h>

#include "ptx.cuh"

namespace dkv {

namespace {

// Eight consecutive values as four f32x2 pairs: (0, 2), (4, 6), (1, 3), (5, 7).  That order costs
// nothing to form from bf16 words, and both pairings of the rotation are then element-wise.
struct Vec8 {
  float2 v[4];
};
__host__ __device__ constexpr int vec8_at(int d) { return (d & ~7) | ((d & 7) >> 1) | ((d & 1) << 2); }

__device__ __forceinline__ Vec8 unpack8(const uint4& w) {
  auto lo = [](uint32_t x) { return __uint_as_float(x << 16); };
  auto hi = [](uint32_t x) { return __uint_as_float(x & 0xffff0000u); };
  Vec8 r;
  r.v[0] = make_float2(lo(w.x), lo(w.y));
  r.v[1] = make_float2(lo(w.z), lo(w.w));
  r.v[2] = make_float2(hi(w.x), hi(w.y));
  r.v[3] = make_float2(hi(w.z), hi(w.w));
  return r;
}
__device__ __forceinline__ uint4 pack8(const Vec8& r) {
  uint4 w;
  __nv_bfloat162* h = reinterpret_cast<__nv_bfloat162*>(&w);
  h[0] = __floats2bfloat162_rn(r.v[0].x, r.v[2].x);
  h[1] = __floats2bfloat162_rn(r.v[0].y, r.v[2].y);
  h[2] = __floats2bfloat162_rn(r.v[1].x, r.v[3].x);
  h[3] = __floats2bfloat162_rn(r.v[1].y, r.v[3].y);
  return w;
}
__device__ __forceinline__ Vec8 load8(const float* p, const float* q) {  // 4 floats each
  const float4 a = *reinterpret_cast<const float4*>(p), b = *reinterpret_cast<const float4*>(q);
  return Vec8{{make_float2(a.x, a.y), make_float2(a.z, a.w), make_float2(b.x, b.y), make_float2(b.z, b.w)}};
}

// Place of value d of n in shared memory: the first four of every Vec8, then the last four, so that
// neighbouring lanes read neighbouring 16 bytes.
__device__ __forceinline__ int split_at(int d, int n) {
  const int p = vec8_at(d) & 7;
  return (p < 4 ? 0 : n / 2) + (d >> 3) * 4 + (p & 3);
}

// Where a lane's vectors A and B lie in a head, and the angles that turn them: 4 from ja
// and 4 from jb on (both of no use where the lane's values are not turned).  In both layouts
// neighbouring lanes read neighbouring vectors.
struct LaneMap {
  int a, b, ja, jb;
  bool ta, tb;
};

template <int D>
__device__ __forceinline__ LaneMap lane_map(int i, int half, bool inter) {
  if (inter) return LaneMap{8 * i, D / 2 + 8 * i, 4 * i, D / 4 + 4 * i, 4 * i < half, D / 4 + 4 * i < half};
  if (8 * i < half) return LaneMap{8 * i, half + 8 * i, 4 * i, half / 2 + 4 * i, true, true};
  return LaneMap{half + 8 * i, D / 2 + 8 * i, 0, 0, false, false};  // behind the turned 2 half values
}

// Frequencies as fractions of a turn in 64-bit fixed point: a row's angle is then
// position * frequency in integer arithmetic, whose overflow drops whole turns.  f / 2 pi
// comes from fp64 once per block; the error of the angle is below 2^-32 turns plus 2^-53 of it.
__device__ __forceinline__ uint64_t turn_fraction(float f) {
  double t = (double)f * 0.15915494309189533577;
  t -= floor(t);
  return (uint64_t)__double2ull_rd(t * 18446744073709551616.0);  // t < 1; 2^64 itself saturates
}

// A lane's cosines and sines, in the order of its values; neg = -sn.
struct Angles {
  Vec8 cs, sn, neg;
};

// The lane's own cosines and sines of its warp's row (1 and 0 where its values are not turned).
__device__ __forceinline__ Angles lane_angles(const float* wc, const float* ws, const LaneMap& m) {
  Angles r{load8(wc + m.ja, wc + m.jb), load8(ws + m.ja, ws + m.jb), {}};
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    if (!(e < 2 ? m.ta : m.tb)) {
      r.cs.v[e] = make_float2(1.f, 1.f);
      r.sn.v[e] = make_float2(0.f, 0.f);
    }
    r.neg.v[e] = make_float2(-r.sn.v[e].x, -r.sn.v[e].y);
  }
  return r;
}

// The warp's cosines and sines of one row in shared memory, then the lane's own of them.
__device__ __forceinline__ Angles row_angles(int p, const uint64_t* freq, int half, float* wc, float* ws, int lane,
                                             const LaneMap& m, bool inter) {
  __syncwarp();
  for (int j = lane; j < half; j += 32) {
    const int turns = (int)(uint32_t)(((uint64_t)(uint32_t)p * freq[j]) >> 32);
    const int at = inter ? j : split_at(j, half);
    sincospif((float)turns * 4.656612873077393e-10f, ws + at, wc + at);  // 2^-31: half turns
  }
  __syncwarp();
  return lane_angles(wc, ws, m);
}

// (u, v) <- (u c - v s, v c + u s)
__device__ __forceinline__ void turn2(float2& u, float2& v, float2 c, float2 s, float2 neg) {
  const float2 x = ffma2(v, neg, fmul2(u, c));
  v = ffma2(u, s, fmul2(v, c));
  u = x;
}
__device__ __forceinline__ void rotate(Vec8& a, Vec8& b, const Vec8& c, const Vec8& s, const Vec8& neg, bool inter) {
  if (inter) {
    turn2(a.v[0], a.v[2], c.v[0], s.v[0], neg.v[0]);
    turn2(a.v[1], a.v[3], c.v[1], s.v[1], neg.v[1]);
    turn2(b.v[0], b.v[2], c.v[2], s.v[2], neg.v[2]);
    turn2(b.v[1], b.v[3], c.v[3], s.v[3], neg.v[3]);
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e) turn2(a.v[e], b.v[e], c.v[e], s.v[e], neg.v[e]);
  }
}

template <int G>
__device__ __forceinline__ float group_sum(float2 p) {
  float v = p.x + p.y;
#pragma unroll
  for (int o = G / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// cp.async: each lane copies the vectors that it will use itself into its own slots of a ring
// in shared memory, some steps ahead of their use, so enough bytes are in flight without
// holding registers and without any barrier.
__device__ __forceinline__ void copy16(void* dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(dst)), "l"(src) : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copies_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

}  // namespace

}  // namespace dkv
