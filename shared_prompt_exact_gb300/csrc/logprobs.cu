// logprobs.cu -- log-probabilities and entropies of the response tokens from the
// logits of the packed rows, and the gradient of the logits.
//
// The logits' rows are the packed rows that predict a response token: the
// prompt's last row (local row 0, when there is a prompt) and the response rows
// after it.  Response token i is predicted by the row before it in its own
// sequence: local row 0 if it opens its segment, else the row of token i - 1.  So
// local row 0 predicts one token per segment and its gradient is the sum over
// the segments, and the last row of each segment predicts nothing.
//
//   z = scale * logits,  lse = log sum_v exp z_v,  p = exp(z - lse)
//   logp_i = z[tok_i] - lse,   H = lse - sum_v p_v z_v
//   dlogits_v = scale * sum_i [ g_i (1[v = tok_i] - p_v) - h_i p_v (z_v - lse + H) ]
//
// Forward: one pass over a row with a running maximum, sum and (for H) weighted
// sum; reads each logit once.  Backward: one pass, reads each logit and writes
// each gradient once.  Statistics are fp32.  Both are bound by HBM bandwidth, given
// enough loads in flight and few instructions per logit: batches of 8 (forward) and 4
// vectors per thread, bf16 maxima two at a time, sums on f32x2 pairs.  Measured at
// 131,072 bf16 logits a row: 17,096 rows with entropies 620 us (7.2 TB/s read, 1.06 of the
// measured copy bandwidth; one vector at a time 841 us), the gradient of 10,479 rows with
// entropies 780 us (6.9 TB/s, 1.01; one vector at a time 883 us).
#include <cooperative_groups.h>
#include <cuda_bf16.h>
#include <math_constants.h>

#include <cfloat>

#include "kernels.h"
#include "ptx.cuh"
#include "segs.cuh"

namespace dkv {

namespace {

namespace cg = cooperative_groups;

constexpr int kLogpThreads = 256;
constexpr int kFwdBatch = 8, kBwdBatch = 4;  // vectors that a thread has in flight
constexpr int kMaxParts = 8;                 // blocks of a forward cluster
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
// Bound on exponents that are multiplied with their power, which is 0 long before (from -126 in base 2 on), so that
// a masked entry adds 0 and not 0 * inf: near enough to 0 that its products with a row's sum or an upstream
// gradient stay finite too.
constexpr float kFloor = -1e4f;

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ float to_f(float x) { return x; }
__device__ __forceinline__ float to_f(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ void from_f(float x, float* d) { *d = x; }
__device__ __forceinline__ void from_f(float x, __nv_bfloat16* d) { *d = __float2bfloat16_rn(x); }

// A vector's values as f32x2 pairs (bf16: neighbours, fp32: neighbours).
__device__ __forceinline__ void unpack(const uint4& v, float2 (&f)[2]) {
  f[0] = make_float2(__uint_as_float(v.x), __uint_as_float(v.y));
  f[1] = make_float2(__uint_as_float(v.z), __uint_as_float(v.w));
}
__device__ __forceinline__ void unpack(const uint4& v, float2 (&f)[4]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int e = 0; e < 4; ++e) f[e] = make_float2(__uint_as_float(w[e] << 16), __uint_as_float(w[e] & 0xffff0000u));
}
__device__ __forceinline__ uint4 pack(const float2 (&f)[2]) {
  return make_uint4(__float_as_uint(f[0].x), __float_as_uint(f[0].y), __float_as_uint(f[1].x), __float_as_uint(f[1].y));
}
__device__ __forceinline__ uint4 pack(const float2 (&f)[4]) {
  uint4 v;
  __nv_bfloat162* h = reinterpret_cast<__nv_bfloat162*>(&v);
#pragma unroll
  for (int e = 0; e < 4; ++e) h[e] = __floats2bfloat162_rn(f[e].x, f[e].y);
  return v;
}

// Largest value of K vectors; a NaN does not count.
template <int K>
__device__ __forceinline__ float max_of(const uint4 (&v)[K], float) {
  float m = -CUDART_INF_F;
#pragma unroll
  for (int k = 0; k < K; ++k) {
    m = fmax3(m, __uint_as_float(v[k].x), __uint_as_float(v[k].y));
    m = fmax3(m, __uint_as_float(v[k].z), __uint_as_float(v[k].w));
  }
  return m;
}
template <int K>
__device__ __forceinline__ float max_of(const uint4 (&v)[K], __nv_bfloat16) {
  __nv_bfloat162 m = __halves2bfloat162(__ushort_as_bfloat16(0xff80), __ushort_as_bfloat16(0xff80));
#pragma unroll
  for (int k = 0; k < K; ++k) {
    const __nv_bfloat162* h = reinterpret_cast<const __nv_bfloat162*>(&v[k]);
    m = __hmax2(m, __hmax2(__hmax2(h[0], h[1]), __hmax2(h[2], h[3])));
  }
  return fmaxf(__low2float(m), __high2float(m));
}

// A 16-byte load that does not stay in L1 (every logit is read once).
__device__ __forceinline__ uint4 load_once(const uint4* p) {
  uint4 v;
  asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p)
               : "memory");
  return v;
}

// The 16-byte vectors of `n` values: [head, head + nv * E), between two ragged ends.
template <typename T>
struct RowVectors {
  static constexpr int E = 16 / sizeof(T);
  int head, nv, tail, ends;  // tail: first element behind the vectors; ends: elements outside them
  __device__ __forceinline__ RowVectors(const T* row, int n) {
    head = (int)(((16 - (reinterpret_cast<uintptr_t>(row) & 15)) & 15) / sizeof(T));
    head = head < n ? head : n;
    nv = (n - head) / E;
    tail = head + nv * E;
    ends = head + n - tail;
  }
  __device__ __forceinline__ int end(int k) const { return k < head ? k : tail + k - head; }
};

// Columns [lo, hi) of part `r` of `parts` of a row: whole vectors, with a ragged end at the row's.
template <typename T>
__device__ __forceinline__ void part_of(const T* row, int V, int r, int parts, int* lo, int* hi) {
  const RowVectors<T> v(row, V);
  *lo = r == 0 ? 0 : v.head + (int)((int64_t)v.nv * r / parts) * RowVectors<T>::E;
  *hi = r == parts - 1 ? V : v.head + (int)((int64_t)v.nv * (r + 1) / parts) * RowVectors<T>::E;
}

// The token that a row other than the prompt's last one predicts: its index, or -1.
// `open` is the index of a segment-opening token that no row predicts (P = 0) and that
// this row's block therefore has to fill in, or -1.
template <int CAP>
__device__ __forceinline__ int predicted(const SegTable<CAP>& seg, int64_t row, int* open) {
  const int n = seg.off[seg.N];
  const int i = (int)row + (seg.P > 0 ? 0 : 1);
  *open = -1;
  if (i >= n) return -1;
  if (seg.off[seg_of(seg, i)] != i) return i;
  if (seg.P == 0) *open = i;
  return -1;
}

// A token's vocabulary entry, or -1 if it is ignored; one past the vocabulary is
// recorded in the status word and ignored.
__device__ __forceinline__ int token_at(const LogpArgs& A, int i) {
  const int64_t t = A.tokens[i];
  if (t < 0) return -1;
  if (t >= A.V) {
    atomicOr(A.status, kDevErrBounds);
    return -1;
  }
  return (int)t;
}

// Running maximum m of the raw logits, sum s of e = 2^((z - m) c) and sum t of e (z - m) c,
// where c = scale log2(e), each as two partial sums.  While only -inf has been seen m is -inf
// and s, t are 0 (NaN after a NaN).
struct Running {
  float m;
  float2 s, t;
};

__device__ __forceinline__ Running nothing_yet() {
  return Running{-CUDART_INF_F, make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
}

// 0 in place of a maximum of -inf.
__device__ __forceinline__ float floor_of(float m) { return m == -CUDART_INF_F ? 0.f : m; }

// Moves (s, t) from their maximum to a larger one.
__device__ __forceinline__ void rebase(Running& r, float m, float c) {
  if (r.m != -CUDART_INF_F) {
    // the bound keeps a maximum that is the type's lowest value, or one below +inf, from leaving 0 * inf
    const float d = fmaxf((r.m - floor_of(m)) * c, kFloor), f = ex2(d);
    r.t = fmul2(ffma2(make_float2(d, d), r.s, r.t), make_float2(f, f));
    r.s = fmul2(r.s, make_float2(f, f));
  }
  r.m = m;
}

__device__ __forceinline__ Running join(Running a, Running b, float c) {
  const float m = fmaxf(a.m, b.m);
  rebase(a, m, c);
  rebase(b, m, c);
  return Running{m, fadd2(a.s, b.s), fadd2(a.t, b.t)};
}

// Adds pairs of values no larger than r.m.
template <bool ENT, int K>
__device__ __forceinline__ void accumulate(Running& r, const float2 (&z)[K], float c) {
  const float base = floor_of(r.m);
  const float2 b2 = make_float2(base, base), c2 = make_float2(c, c);
#pragma unroll
  for (int e = 0; e < K; ++e) {
    // subtracted first: exactly 0 at the maximum, whatever its size
    float2 y = fmul2(fsub2(z[e], b2), c2);
    const float2 x = make_float2(ex2(y.x), ex2(y.y));
    r.s = fadd2(r.s, x);
    if (ENT) {
      y = make_float2(fmaxf(y.x, kFloor), fmaxf(y.y, kFloor));  // a masked logit adds 0, not 0 * inf
      r.t = ffma2(x, y, r.t);
    }
  }
}

template <typename T, bool ENT, int K>
__device__ __forceinline__ void absorb(Running& r, const uint4 (&v)[K], float c) {
  const float m = max_of(v, T());
  if (m > r.m) rebase(r, m, c);
#pragma unroll
  for (int k = 0; k < K; ++k) {
    float2 z[RowVectors<T>::E / 2];
    unpack(v[k], z);
    accumulate<ENT>(r, z, c);
  }
}

__device__ __forceinline__ Running warp_join(Running r, float c) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    Running b;
    b.m = __shfl_xor_sync(0xffffffffu, r.m, o);
    b.s = make_float2(__shfl_xor_sync(0xffffffffu, r.s.x, o), 0.f);
    b.t = make_float2(__shfl_xor_sync(0xffffffffu, r.t.x, o), 0.f);
    r = join(r, b, c);
  }
  return r;
}

// The block's sums, in its first warp (in the x halves).
__device__ __forceinline__ Running block_join(Running r, float c) {
  __shared__ Running part[kLogpThreads / 32];
  r.s = make_float2(r.s.x + r.s.y, 0.f);
  r.t = make_float2(r.t.x + r.t.y, 0.f);
  r = warp_join(r, c);
  if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = r;
  __syncthreads();
  if (threadIdx.x >= 32) return r;
  return warp_join(threadIdx.x < kLogpThreads / 32 ? part[threadIdx.x] : nothing_yet(), c);
}

// One row per cluster of `parts` blocks (a part of the columns each), joined by its first block.
template <typename T, bool ENT, int CAP>
__global__ void __launch_bounds__(kLogpThreads, 4) logp_fwd_kernel(const LogpArgs A, int parts,
                                                                   const __grid_constant__ SegTable<CAP> seg) {
  constexpr int U = kFwdBatch;
  const int64_t row = blockIdx.x / parts;
  const int rank = blockIdx.x % parts, n = seg.off[seg.N], tid = threadIdx.x;
  const bool shared_row = seg.P > 0 && row == 0;
  int open = -1, mine = -1, live = 0;
  if (shared_row) {
    for (int s = tid; s < seg.N; s += kLogpThreads)
      if (seg.off[s] < seg.off[s + 1] && token_at(A, seg.off[s]) >= 0) live = 1;
    live = __syncthreads_or(live);
  } else {
    mine = predicted(seg, row, &open);
    if (mine >= 0) live = token_at(A, mine) >= 0;
    if (seg.P == 0 && row == 0 && rank == 0 && tid == 0 && n > 0) {  // token 0 opens its segment
      A.logp[0] = 0.f;
      if (ENT) A.entropy[0] = 0.f;
    }
  }
  if (!live) {  // the same in all blocks of the row
    if (rank) return;
    if (shared_row) {
      for (int s = tid; s < seg.N; s += kLogpThreads)
        if (seg.off[s] < seg.off[s + 1]) {
          A.logp[seg.off[s]] = 0.f;
          if (ENT) A.entropy[seg.off[s]] = 0.f;
        }
    } else if (tid == 0 && (mine >= 0 || open >= 0)) {
      A.logp[mine >= 0 ? mine : open] = 0.f;
      if (ENT) A.entropy[mine >= 0 ? mine : open] = 0.f;
    }
    if (tid == 0 && A.lse) A.lse[row] = 0.f;
    return;
  }
  const float c = A.scale * kLog2e;
  const T* x = static_cast<const T*>(A.logits) + row * A.stride;
  int lo, hi;
  part_of(x, A.V, rank, parts, &lo, &hi);
  const RowVectors<T> v(x + lo, hi - lo);
  Running r = nothing_yet();
  const uint4* xv = reinterpret_cast<const uint4*>(x + lo + v.head);
  int k = tid;
  for (; k + (U - 1) * kLogpThreads < v.nv; k += U * kLogpThreads) {
    uint4 w[U];
#pragma unroll
    for (int u = 0; u < U; ++u) w[u] = load_once(xv + k + u * kLogpThreads);
    absorb<T, ENT>(r, w, c);
  }
  for (; k < v.nv; k += kLogpThreads) {
    const uint4 w[1] = {load_once(xv + k)};
    absorb<T, ENT>(r, w, c);
  }
  for (k = tid; k < v.ends; k += kLogpThreads) {
    const float2 z[1] = {make_float2(to_f(x[lo + v.end(k)]), -CUDART_INF_F)};
    if (z[0].x > r.m) rebase(r, z[0].x, c);
    accumulate<ENT>(r, z, c);
  }
  r = block_join(r, c);
  if (parts > 1) {
    __shared__ Running joined[kMaxParts];
    cg::cluster_group cluster = cg::this_cluster();
    cluster.sync();  // the first block has to run before its memory is written
    if (tid == 0) *cluster.map_shared_rank(&joined[rank], 0) = r;
    cluster.sync();
    if (rank) return;
    if (tid < 32) r = warp_join(tid < parts ? joined[tid] : nothing_yet(), c);
  }
  // the first warp has the row's sums; s is 0 only in a row that is -inf throughout: lse and logp
  // are -inf there, H is 0
  if (tid >= 32) return;
  const bool none = r.s.x == 0.f;
  const float ln_sum = logf(r.s.x), ent = none ? 0.f : ln_sum - r.t.x / r.s.x * kLn2;
  auto write = [&](int i) {
    const int tok = token_at(A, i);
    // smaller terms than z - lse, so a likelier token keeps more digits
    const float lp = tok < 0 ? 0.f : none ? -CUDART_INF_F : (to_f(x[tok]) - r.m) * A.scale - ln_sum;
    A.logp[i] = lp;
    if (ENT) A.entropy[i] = tok < 0 ? 0.f : ent;
  };
  if (shared_row) {
    for (int s = tid; s < seg.N; s += 32)
      if (seg.off[s] < seg.off[s + 1]) write(seg.off[s]);
  } else if (tid == 0) {
    write(mine);
  }
  // scale * max may pass fp32's range in a row of the type's lowest or largest values: its lse stays finite, so
  // that -inf means a row without entries and nothing else
  if (tid == 0 && A.lse) {
    const float lse = fmaf(r.m, A.scale, ln_sum);
    A.lse[row] = none ? -CUDART_INF_F : isinf(lse) ? copysignf(FLT_MAX, lse) : lse;
  }
}

__device__ __forceinline__ float block_sum(float v) {
  __shared__ float part[kLogpThreads / 32];
  __syncthreads();
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = v;
  __syncthreads();
  v = 0.f;
  for (int k = 0; k < kLogpThreads / 32; ++k) v += part[k];
  return v;
}

// A row's gradient p (k0 + k1 d), d = z scale - lse, p = e^d for a raw logit z.  d is formed
// before the scaling to base 2, so that its rounding is relative to d and not to z.
struct RowGrad {
  float scale, lse, k0, k1;
  float base;  // subtracted from z first, in rows that are summed again; else 0
};
template <bool ENT>
__device__ __forceinline__ float2 grad_of(float2 z, const RowGrad& r) {
  z = fsub2(z, make_float2(r.base, r.base));
  const float2 d = ffma2(z, make_float2(r.scale, r.scale), make_float2(-r.lse, -r.lse));
  const float2 y = fmul2(d, make_float2(kLog2e, kLog2e)), p = make_float2(ex2(y.x), ex2(y.y));
  const float2 k = make_float2(r.k0, r.k0);
  if (!ENT) return fmul2(p, k);
  return fmul2(p, ffma2(make_float2(fmaxf(d.x, kFloor), fmaxf(d.y, kFloor)), make_float2(r.k1, r.k1), k));
}
template <bool ENT>
__device__ __forceinline__ float grad_of(float z, const RowGrad& r) {
  const float d = fmaf(z - r.base, r.scale, -r.lse), p = ex2(d * kLog2e);
  return ENT ? p * fmaf(fmaxf(d, kFloor), r.k1, r.k0) : p * r.k0;
}

// Slots for the keys of N segments.
__host__ __device__ __forceinline__ int key_slots(int N) {
  int n2 = 2;
  while (n2 < N) n2 <<= 1;
  return n2;
}

// The shared row's targets as keys (token, segment), ascending, those that are ignored last.
constexpr uint64_t kNoKey = ~0ull;

// Sorts n2 = 2^k keys, then sums the gradients of equal tokens: at the last key of a token `sum` gets
// them all, added in an order that depends on the keys alone.  `sum` and `spare` hold n2 values
// each; returns the one that has the sums.  Up to a key per thread each key counts those before it;
// more are sorted by a bitonic network (a call with 4,095 segments: 166 us, 546 when every pair of
// targets was compared; with 256: 11.1 us by counting, 12.8 by the network).
template <int CAP>
__device__ __noinline__ float* sum_targets(const LogpArgs& A, const SegTable<CAP>& seg, uint64_t* key, float* sum,
                                           float* spare, int n2) {
  const int tid = threadIdx.x;
  __syncthreads();
  if (n2 <= kLogpThreads) {
    const uint64_t mine = tid < n2 ? key[tid] : kNoKey;
    int rank = 0;
    for (int u = 0; u < n2; ++u) rank += key[u] < mine || (key[u] == mine && u < tid);
    __syncthreads();
    if (tid < n2) key[rank] = mine;
    __syncthreads();
  }
  for (int k = 2; k <= n2 && n2 > kLogpThreads; k <<= 1)
    for (int j = k >> 1; j > 0; j >>= 1) {
      for (int i = tid; i < n2; i += kLogpThreads) {
        const int p = i ^ j;
        if (p > i && (key[i] > key[p]) == ((i & k) == 0)) {
          const uint64_t t = key[i];
          key[i] = key[p];
          key[p] = t;
        }
      }
      __syncthreads();
    }
  for (int i = tid; i < n2; i += kLogpThreads) sum[i] = key[i] == kNoKey ? 0.f : A.dlogp[seg.off[(uint32_t)key[i]]];
  __syncthreads();
  for (int d = 1; d < n2; d <<= 1) {
    for (int i = tid; i < n2; i += kLogpThreads)
      spare[i] = sum[i] + (i >= d && (key[i] >> 32) == (key[i - d] >> 32) ? sum[i - d] : 0.f);
    __syncthreads();
    float* t = sum;
    sum = spare;
    spare = t;
  }
  return sum;
}

// The rounding of an fp32 lse, half a step of its binade, is a relative error of every probability of its row, and as
// much of g at a target, whose g (1 - p) may be far smaller.  Up to this |lse| it is taken as it is: half a step is
// 2^-18 below 128, for fp32 logits no more than a sum may be off, and 2^-15 below 1,024, for bf16 a 64th of the half
// step that each gradient is then rounded by.  In rows further from 0 a block forms the sum again, apart from the maximum, before it or anyone
// overwrites the row, and takes the whole row: 8,000 rows of 131,072 bf16 take 921 us instead of 608, 3,000 of fp32
// 709 instead of 454, 20 rows of bf16 24 instead of 4.7 (in a graph).
template <typename T>
__device__ constexpr float lse_holds() {
  return sizeof(T) == 4 ? 128.f : 1024.f;
}

// A row's maximum, and the logarithm of its sum relative to that, in every thread of the block.
template <typename T>
__device__ __noinline__ float2 row_sum(const T* x, int V, float c) {
  constexpr int U = kBwdBatch;
  __shared__ Running sums;
  const int tid = threadIdx.x;
  const RowVectors<T> v(x, V);
  const uint4* xv = reinterpret_cast<const uint4*>(x + v.head);
  Running r = nothing_yet();
  int k = tid;
  for (; k + (U - 1) * kLogpThreads < v.nv; k += U * kLogpThreads) {
    uint4 w[U];
#pragma unroll
    for (int u = 0; u < U; ++u) w[u] = load_once(xv + k + u * kLogpThreads);
    absorb<T, false>(r, w, c);
  }
  for (; k < v.nv; k += kLogpThreads) {
    const uint4 w[1] = {load_once(xv + k)};
    absorb<T, false>(r, w, c);
  }
  for (k = tid; k < v.ends; k += kLogpThreads) {
    const float2 z[1] = {make_float2(to_f(x[v.end(k)]), -CUDART_INF_F)};
    if (z[0].x > r.m) rebase(r, z[0].x, c);
    accumulate<false>(r, z, c);
  }
  r = block_join(r, c);
  if (tid == 0) sums = r;
  __syncthreads();
  return make_float2(sums.m, logf(sums.s.x));
}

// Block (row, part): one part of one row's columns.
template <typename T, bool ENT, int CAP>
__global__ void __launch_bounds__(kLogpThreads, 5) logp_bwd_kernel(const LogpArgs A, int parts,
                                                                   const __grid_constant__ SegTable<CAP> seg) {
  constexpr int P2 = RowVectors<T>::E / 2, U = kBwdBatch;
  extern __shared__ uint64_t keys[];  // the shared row's targets: n2 keys, then two values for each
  const int64_t row = blockIdx.x / parts;
  const int tid = threadIdx.x;
  const bool shared_row = seg.P > 0 && row == 0;
  const T* x = static_cast<const T*>(A.logits) + row * A.stride;
  T* y = static_cast<T*>(A.dlogits) + row * A.dstride;
  int lo, hi;
  part_of(y, A.V, (int)(blockIdx.x % parts), parts, &lo, &hi);
  const float lse = A.lse[row];
  const bool renew = fabsf(lse) > lse_holds<T>() && lse != -CUDART_INF_F;
  if (renew) {  // the first block takes the whole row, whose sum it has to form before anyone overwrites it
    if (blockIdx.x % parts) return;
    lo = 0;
    hi = A.V;
  }
  float g = 0.f, h = 0.f, ent = 0.f;
  int tok = -1;
  bool flows;
  const int n2 = key_slots(seg.N);
  if (shared_row) {
    int any = -1;
    bool targets = false;  // gradients that cancel in g still reach their targets
    for (int s = tid; s < n2; s += kLogpThreads) {
      const int i = s < seg.N ? seg.off[s] : 0;
      const int t = s < seg.N && i < seg.off[s + 1] ? token_at(A, i) : -1;
      keys[s] = t >= 0 ? (uint64_t)t << 32 | (uint32_t)s : kNoKey;
      if (t >= 0) {
        const float gi = A.dlogp[i];
        targets |= gi != 0.f;
        g += gi;
        if (ENT) h += A.dentropy[i];
        any = i;
      }
    }
    g = block_sum(g);
    if (ENT) {
      h = block_sum(h);
      // every live token of the row has the row's entropy: take the last one's
      __shared__ int last;
      if (tid == 0) last = -1;
      __syncthreads();
      if (any >= 0) atomicMax(&last, any);
      __syncthreads();
      ent = last >= 0 ? A.entropy[last] : 0.f;
    }
    flows = __syncthreads_or(targets) || h != 0.f;
  } else {
    int open;
    const int i = predicted(seg, row, &open);
    if (i >= 0) {  // all at once; an ignored token's values count for nothing
      g = A.dlogp[i];
      if (ENT) {
        h = A.dentropy[i];
        ent = A.entropy[i];
      }
      tok = token_at(A, i);
      if (tok < 0) g = h = 0.f;
    }
    flows = g != 0.f || h != 0.f;
  }
  const RowVectors<T> v(y + lo, hi - lo);
  uint4* yv = reinterpret_cast<uint4*>(y + lo + v.head);
  if (!flows || lse == -CUDART_INF_F) {
    // nothing flows into this row (or it is masked throughout): zeros, without reading it
    for (int k = tid; k < v.nv; k += kLogpThreads) yv[k] = make_uint4(0, 0, 0, 0);
    for (int k = tid; k < v.ends; k += kLogpThreads) from_f(0.f, y + lo + v.end(k));
    return;
  }
  const float scale = A.scale;
  RowGrad rg{scale, lse, -scale * fmaf(h, ent, g), -scale * h, 0.f};
  if (renew) {
    const float2 sum = row_sum(x, A.V, scale * kLog2e);
    rg.base = sum.x;
    rg.lse = sum.y;
  }
  auto here = [&](int t) { return t >= lo && t < hi; };  // targets in this block's columns
  // The targets' gradients, from logits that an in-place pass is about to overwrite; in the shared
  // row one for each token, at the last of its keys.
  float vt = 0.f;
  float* s_v = reinterpret_cast<float*>(keys + n2);
  auto last_key = [&](int i) {
    return keys[i] != kNoKey && (i == n2 - 1 || (keys[i] >> 32) != (keys[i + 1] >> 32)) && here((int)(keys[i] >> 32));
  };
  if (shared_row) {
    s_v = sum_targets(A, seg, keys, s_v, s_v + n2, n2);
    for (int i = tid; i < n2; i += kLogpThreads)
      if (last_key(i)) s_v[i] = fmaf(scale, s_v[i], grad_of<ENT>(to_f(x[keys[i] >> 32]), rg));
  } else if (tid == 0 && here(tok)) {
    vt = fmaf(scale, g, grad_of<ENT>(to_f(x[tok]), rg));
  }
  // needed in place only, but the other calls keep it too: without it the block's warps drift apart
  // and 10,479 rows of 131,072 bf16 take 826 us instead of 779
  __syncthreads();
  if (((reinterpret_cast<uintptr_t>(x) ^ reinterpret_cast<uintptr_t>(y)) & 15) == 0) {
    const uint4* xv = reinterpret_cast<const uint4*>(x + lo + v.head);
    auto grads = [&](const uint4& w) {
      float2 z[P2];
      unpack(w, z);
#pragma unroll
      for (int e = 0; e < P2; ++e) z[e] = grad_of<ENT>(z[e], rg);
      return pack(z);
    };
    int k = tid;
    for (; k + (U - 1) * kLogpThreads < v.nv; k += U * kLogpThreads) {
      uint4 w[U];
#pragma unroll
      for (int u = 0; u < U; ++u) w[u] = load_once(xv + k + u * kLogpThreads);
#pragma unroll
      for (int u = 0; u < U; ++u) yv[k + u * kLogpThreads] = grads(w[u]);
    }
    for (; k < v.nv; k += kLogpThreads) yv[k] = grads(load_once(xv + k));
    for (k = tid; k < v.ends; k += kLogpThreads) {
      const int j = lo + v.end(k);
      from_f(grad_of<ENT>(to_f(x[j]), rg), y + j);
    }
  } else {
    // rows that start at different offsets within 16 bytes: 8,000 rows of 131,071 bf16 at strides of 131,136 and
    // 131,135 take 2,450 us, at equal ones 623; 4,000 of 128,255 fp32 1,270 and 698
#pragma unroll 4
    for (int j = lo + tid; j < hi; j += kLogpThreads) from_f(grad_of<ENT>(to_f(x[j]), rg), y + j);
  }
  __syncthreads();
  if (shared_row) {
    for (int i = tid; i < n2; i += kLogpThreads)
      if (last_key(i)) from_f(s_v[i], y + (keys[i] >> 32));
  } else if (tid == 0 && here(tok)) {
    from_f(vt, y + tok);
  }
}

// Blocks per row of the forward: one where the rows fill the GPU, else up to a cluster, which costs
// a join.  At 131,072 bf16 logits: 80 rows 14.5 us in parts, 19.6 whole (cold, launch included);
// 320 rows 26 us whole, 30 in parts.
int fwd_parts(int64_t rows, int64_t bytes) {
  int parts = 1;
  while (parts < kMaxParts && rows * parts * 2 <= 608 && bytes / (parts * 2) >= 32768) parts *= 2;
  return parts;
}

// Blocks per row of the backward, which nothing has to join: parts of 64 KB, which leave a shorter
// last round of blocks than whole rows (10,479 rows of 256 KB: 782 us, whole 808, parts of 16 KB
// 900), and of 16 KB where even those are few (20 rows: 11.4 us against 13.4).
int bwd_parts(int64_t rows, int64_t bytes) {
  const int64_t parts = (bytes + 65535) / 65536;
  return (int)(rows * parts < 608 ? (bytes + 16383) / 16384 : parts);
}

template <typename T, bool ENT, int CAP>
cudaError_t launch_logp_c(bool backward, const LogpArgs& a, int P, int N, const int32_t* off, cudaStream_t st) {
  const SegTable<CAP> s = make_segs<CAP>(P, N, off);
  const int64_t rows = off[N] + (P > 0 ? 1 : 0);
  const int64_t bytes = (int64_t)a.V * sizeof(T);
  const int parts = backward ? bwd_parts(rows, bytes) : fwd_parts(rows, bytes);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(rows * parts));
  cfg.blockDim = dim3(kLogpThreads);
  cfg.stream = st;
  if (!backward) {
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = parts;
    attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = parts > 1 ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, logp_fwd_kernel<T, ENT, CAP>, a, parts, s);
  }
  cfg.dynamicSmemBytes = P > 0 ? (size_t)key_slots(N) * 16 : 0;
  if (cfg.dynamicSmemBytes > 32768) {  // beyond 48 KB with the kernel's static arrays
    const cudaError_t e = cudaFuncSetAttribute(logp_bwd_kernel<T, ENT, CAP>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               key_slots(kMaxSegs) * 16);
    if (e != cudaSuccess) return e;
  }
  return cudaLaunchKernelEx(&cfg, logp_bwd_kernel<T, ENT, CAP>, a, parts, s);
}

template <typename T, bool ENT>
cudaError_t launch_logp_e(bool backward, const LogpArgs& a, int P, int N, const int32_t* off, cudaStream_t st) {
  return N <= kSmallSegs ? launch_logp_c<T, ENT, kSmallSegs>(backward, a, P, N, off, st)
                         : launch_logp_c<T, ENT, kMaxSegs>(backward, a, P, N, off, st);
}

template <typename T>
cudaError_t launch_logp_t(bool backward, const LogpArgs& a, int P, int N, const int32_t* off, cudaStream_t st) {
  const bool ent = backward ? a.dentropy != nullptr : a.entropy != nullptr;
  return ent ? launch_logp_e<T, true>(backward, a, P, N, off, st) : launch_logp_e<T, false>(backward, a, P, N, off, st);
}

}  // namespace

cudaError_t launch_logprobs(bool backward, bool f32, const LogpArgs& a, int P, int N, const int32_t* off,
                            cudaStream_t st) {
  return f32 ? launch_logp_t<float>(backward, a, P, N, off, st)
             : launch_logp_t<__nv_bfloat16>(backward, a, P, N, off, st);
}

}  // namespace dkv
