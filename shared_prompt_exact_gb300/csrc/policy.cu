// policy.cu -- clipped policy loss with a KL term and an entropy bonus over the
// packed response tokens, and its gradient.
//
// Per live token, with d = logp - old, rho = e^d, x = ref - logp and advantage A:
//   policy = -A min(rho, 1 + hi) for A > 0,  -A max(rho, 1 - lo) for A < 0 (with a dual
//            clip at most -A c),  0 for A = 0
//   kl     = e^x - x - 1
//   loss   = sum_n w_n sum_{live tokens of segment n} (policy + b kl - e H)
//   d loss / d logp = w_n (-A rho [not beyond a bound] - b (e^x - 1)),  d loss / d H = -e w_n
//
// The clip tests compare d with the bounds' logarithms: d exactly, as the fp32 difference
// and its rounding error, with log(1 + hi) and the others as sums of two fp32 values
// from fp64.  So no token changes sides by rounding.
//
// Policy terms of either sign cancel in the sum, so each is summed as -A and -A (ratio - 1): -A is
// exact, ratio - 1 comes from the same series as the KL term, and the sums keep their rounding
// errors beside them.  fp64 would do the same, but its adds run at two lanes per clock and SM
// here: with fp64 trees a call on 4M tokens took 172 us instead of 32.
//
// A block takes up to kPolicyChunk tokens of ONE segment, all of whose loads are issued before
// the first is used, and makes one record of sums; a single block then turns the records into
// weights and the loss in a fixed order.  Blocks are numbered without a list: segment n owns
// blocks [off[n] / chunk + n, off[n + 1] / chunk + n + 1), at least as many as it has chunks.  Up
// to kClusterBlocks blocks run as one cluster whose first block joins the records from its shared
// memory; more write them to the workspace for a second launch.
//
// Up to some 100,000 tokens a call is launch latency (in a graph 4.5 to 5.3 us, the gradients 2 to
// 2.5).  At 4.04M tokens (1,024 responses, every input in use) the forward takes 33 us, 2.6 TB/s,
// 6 of them the join, and the gradients 23 us, 4.5 TB/s.  What bounds them is the shape of the work rather than
// a unit: a block loads one chunk, whose latency only the other blocks of its SM cover, and one block joins
// the records behind all of them.  The arithmetic is a tenth: a cold call without it takes 36 us of 40 (the ALU pipe, which
// has the comparisons and selects around the bounds, is 59 % busy), and doing it on f32x2 pairs of
// tokens took a tenth off both directions.  Four tokens a thread in chunks of
// 1,024 beat eight in 2,048 (40 against 46 us cold): more resident threads outweigh fewer blocks.
// For the same reason blocks that stay and walk several chunks, the next one's loads ahead of the sums, lose:
// 42 against 40 us cold, the gradients 32 against 28, although they make a third of the records.
#include <cooperative_groups.h>
#include <cuda_runtime.h>

#include <utility>

#include "kernels.h"
#include "launch.cuh"
#include "ptx.cuh"
#include "segs.cuh"

namespace dkv {

namespace {

namespace cg = cooperative_groups;

constexpr int kPolicyThreads = 256;
constexpr int kPerThread = kPolicyChunk / kPolicyThreads;
constexpr int kClusterBlocks = 8;

// A sum kept as hi + lo, with the rounding errors of the additions in lo (NaN once hi is not finite).
struct Sum2 {
  float hi, lo;
};
__device__ __forceinline__ Sum2 add(const Sum2& a, const Sum2& b) {
  const float s = a.hi + b.hi, bb = s - a.hi;
  return Sum2{s, (a.hi - (s - bb)) + (b.hi - bb) + (a.lo + b.lo)};
}
__device__ __forceinline__ Sum2 times(float w, const Sum2& v) {
  const float p = w * v.hi;
  return Sum2{p, fmaf(w, v.lo, fmaf(w, v.hi, -p))};
}
__device__ __forceinline__ double value(const Sum2& v) {
  return fabsf(v.hi) <= 3.4e38f ? (double)v.hi + (double)v.lo : (double)v.hi;
}

// A chunk's sums; counts holds the live tokens and, in the upper half, those beyond a bound.
struct alignas(8) Record {
  Sum2 policy;
  float kl, ent;
  uint32_t counts;
  int seg;
};

// The segments of every 2^shift-th block, so that a block finds its own among few.
constexpr int kIndex = 128;
struct BlockIndex {
  int shift;
  uint16_t seg[kIndex + 1];
};

__host__ __device__ __forceinline__ int first_block(int off, int n) { return off / kPolicyChunk + n; }

BlockIndex make_index(int N, const int32_t* off, int blocks) {
  BlockIndex x;
  x.shift = 0;
  while ((blocks - 1) >> x.shift >= kIndex) ++x.shift;
  int n = 0;
  for (int k = 0; k <= kIndex; ++k) {
    const int block = k << x.shift;
    if (block >= blocks) {
      x.seg[k] = (uint16_t)(N - 1);
      break;
    }
    int hi = N - 1;  // the largest segment whose first block is no later
    while (n < hi) {
      const int mid = (n + hi + 1) >> 1;
      if (first_block(off[mid], mid) <= block) n = mid;
      else hi = mid - 1;
    }
    x.seg[k] = (uint16_t)n;
  }
  return x;
}

// The block's segment and its token range [lo, hi) (empty when the segment needs fewer blocks).
struct Chunk {
  int seg, lo, hi;
};
template <int CAP>
__device__ __forceinline__ Chunk chunk_of(const SegTable<CAP>& s, const BlockIndex& x, int block) {
  int lo = x.seg[block >> x.shift], hi = x.shift ? x.seg[(block >> x.shift) + 1] : lo;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (first_block(s.off[mid], mid) <= block) lo = mid;
    else hi = mid - 1;
  }
  const int64_t begin = (int64_t)s.off[lo] + (int64_t)(block - first_block(s.off[lo], lo)) * kPolicyChunk;
  const int end = s.off[lo + 1];
  if (begin >= end) return Chunk{lo, end, end};
  return Chunk{lo, (int)begin, (int)(begin + kPolicyChunk < end ? begin + kPolicyChunk : end)};
}

// Arithmetic below is on pairs of tokens (f32x2).
__device__ __forceinline__ float2 both(float v) { return make_float2(v, v); }
__device__ __forceinline__ float2 pick(bool x, bool y, float a, float b) { return make_float2(x ? a : b, y ? a : b); }

// a - b as the rounded difference and what rounding took away (finite even where the difference is not).
__device__ __forceinline__ float2 exact_diff(float2 a, float2 b, float2* err) {
  const float2 d = fsub2(a, b), bb = fsub2(d, a);
  const float2 e = fsub2(fsub2(a, fsub2(d, bb)), fadd2(b, bb));
  *err = make_float2(fmaxf(e.x, -1e30f), fmaxf(e.y, -1e30f));  // not NaN
  return d;
}
// The sign of (d + e) - t: d - t.hi is exact where the two are close, and elsewhere larger than the rest.
__device__ __forceinline__ float2 beyond(float2 d, float2 e, float2 hi, float2 lo) {
  return fadd2(fsub2(d, hi), fsub2(e, lo));
}

// e^x - x - 1 for |x| < 1 (its series; the difference itself would cancel).
__device__ __forceinline__ float2 series(float2 x) {
  float2 p = both(1.f / 39916800.f);
  p = ffma2(p, x, both(1.f / 3628800.f));
  p = ffma2(p, x, both(1.f / 362880.f));
  p = ffma2(p, x, both(1.f / 40320.f));
  p = ffma2(p, x, both(1.f / 5040.f));
  p = ffma2(p, x, both(1.f / 720.f));
  p = ffma2(p, x, both(1.f / 120.f));
  p = ffma2(p, x, both(1.f / 24.f));
  p = ffma2(p, x, both(1.f / 6.f));
  p = ffma2(p, x, both(0.5f));
  return fmul2(fmul2(p, x), x);
}
__device__ __forceinline__ bool far(float2 x) { return !(fmaxf(fabsf(x.x), fabsf(x.y)) < 1.f); }

// e^x - x - 1 and e^x - 1.
struct Kl {
  float2 kl, slope;
};
__device__ __forceinline__ Kl kl_of(float2 x) {
  Kl r;
  r.kl = series(x);
  r.slope = fadd2(r.kl, x);
  if (far(x)) {
    auto direct = [](float v, float& kl, float& slope) {
      if (fabsf(v) < 1.f) return;
      slope = expf(v) - 1.f;
      kl = slope - v;
    };
    direct(x.x, r.kl.x, r.slope.x);
    direct(x.y, r.kl.y, r.slope.y);
  }
  return r;
}

// Two tokens' bounded ratios as base + v + rest, and whether they are bounds.  base is 1 for a bound
// and a ratio near 1: policy terms of either sign cancel, and A (1 + v + rest) is then summed from A,
// which is exact, and two products of small factors.  A ratio that is far from 1 has base 0.
// Without BOUNDED the ratio is left unbounded (the backward only needs to know).
struct Term {
  float2 base, v, rest;
  bool clipped_x, clipped_y;
};
template <bool BOUNDED>
__device__ __forceinline__ Term term_of(const PolicyArgs& A, float2 logp, float2 old, float2 adv) {
  float2 e;
  const float2 d = exact_diff(logp, old, &e);
  Term t;
  t.base = both(1.f);
  t.v = d;
  t.rest = fadd2(series(d), e);  // e^d - 1 = d + series
  if (far(d)) {
    auto direct = [](float x, float err, float a, float& base, float& v, float& rest) {
      if (fabsf(x) < 1.f) return;
      base = 0.f;
      v = a == 0.f ? 0.f : expf(x);  // not 0 * inf
      rest = fabsf(x) < 80.f ? v * err : 0.f;
    };
    direct(d.x, e.x, adv.x, t.base.x, t.v.x, t.rest.x);
    direct(d.y, e.y, adv.y, t.base.y, t.v.y, t.rest.y);
  }
  const bool gx = adv.x > 0.f, gy = adv.y > 0.f, lx = adv.x < 0.f, ly = adv.y < 0.f;
  const float2 x = beyond(d, e, pick(gx, gy, A.up.hi, A.down.hi), pick(gx, gy, A.up.lo, A.down.lo));
  t.clipped_x = gx ? x.x > 0.f : lx && x.x < 0.f;
  t.clipped_y = gy ? x.y > 0.f : ly && x.y < 0.f;
  bool far_x = false, far_y = false;
  if (A.has_dual) {
    const float2 up = beyond(d, e, both(A.dual.hi), both(A.dual.lo));
    far_x = lx && up.x > 0.f;
    far_y = ly && up.y > 0.f;
  }
  if (BOUNDED) {
    const float2 bv = pick(gx, gy, A.add_up.hi, A.add_down.hi), br = pick(gx, gy, A.add_up.lo, A.add_down.lo);
    if (t.clipped_x) t.base.x = 1.f, t.v.x = bv.x, t.rest.x = br.x;
    if (t.clipped_y) t.base.y = 1.f, t.v.y = bv.y, t.rest.y = br.y;
    if (far_x) t.base.x = 1.f, t.v.x = A.add_dual.hi, t.rest.x = A.add_dual.lo;
    if (far_y) t.base.y = 1.f, t.v.y = A.add_dual.hi, t.rest.y = A.add_dual.lo;
  }
  t.clipped_x |= far_x;
  t.clipped_y |= far_y;
  return t;
}

// A thread's tokens of a chunk, lo + tid + k * threads; FULL: all of them exist.  Masked ones are
// loaded, not used.
struct Tokens {
  float logp[kPerThread], old[kPerThread], adv[kPerThread], ref[kPerThread], ent[kPerThread];
  bool on[kPerThread];
};
template <bool FULL>
__device__ __forceinline__ bool exists(const Chunk& c, int k) {
  return FULL || c.lo + (int)threadIdx.x + k * kPolicyThreads < c.hi;
}
template <bool FULL, bool ENT>
__device__ __forceinline__ void load_tokens(const PolicyArgs& A, const Chunk& c, Tokens& t) {
  const int64_t at = (int64_t)c.lo + threadIdx.x;
  const float *logp = A.logp + at, *old = A.old_logp + at, *ref = A.ref_logp + at, *ent = A.entropy + at;
  const float* adv = A.per_token ? A.adv + at : A.adv + c.seg;
  const uint8_t* mask = A.mask + at;
  const bool per_token = A.per_token, has_ref = A.ref_logp, has_ent = ENT && A.entropy, has_mask = A.mask;
#pragma unroll
  for (int k = 0; k < kPerThread; ++k) {
    t.on[k] = exists<FULL>(c, k);
    t.logp[k] = t.old[k] = t.adv[k] = t.ref[k] = t.ent[k] = 0.f;
    if (FULL || t.on[k]) {
      t.logp[k] = logp[k * kPolicyThreads];
      t.old[k] = old[k * kPolicyThreads];
      t.adv[k] = adv[per_token ? k * kPolicyThreads : 0];
      if (has_ref) t.ref[k] = ref[k * kPolicyThreads];
      if (has_ent) t.ent[k] = ent[k * kPolicyThreads];
      if (has_mask) t.on[k] = mask[k * kPolicyThreads] != 0;
    }
  }
}

__device__ __forceinline__ Sum2 warp_sum(Sum2 v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1)
    v = add(v, Sum2{__shfl_xor_sync(0xffffffffu, v.hi, o), __shfl_xor_sync(0xffffffffu, v.lo, o)});
  return v;
}
// A thread's share of its chunk's sums; policy: of A ratio, whose sign the join turns.
struct Partial {
  Sum2 policy;
  float kl, ent;
  uint32_t counts;
};
template <bool FULL>
__device__ __forceinline__ Partial sum_tokens(const PolicyArgs& A, const Chunk& c) {
  Tokens x;
  load_tokens<FULL, true>(A, c, x);
  const float2 zero = both(0.f);
  float2 hi = zero, lo = zero, kl = zero, ent = zero;
  uint32_t counts = 0;
#pragma unroll
  for (int k = 0; k < kPerThread; k += 2) {
    if (!FULL && c.lo + k * kPolicyThreads >= c.hi) break;  // the same for the whole block
    const float2 logp = make_float2(x.logp[k], x.logp[k + 1]), a = make_float2(x.adv[k], x.adv[k + 1]);
    const Term t = term_of<true>(A, logp, make_float2(x.old[k], x.old[k + 1]), a);
    const float2 p = fmul2(a, t.v), ab = fmul2(a, t.base);
    float2 y = fadd2(ab, p);
    // the errors of the product, of the sum (|v| <= 1 but for bounds above 2), and the rest
    float2 z = ffma2(a, t.rest, fadd2(ffma2(a, t.v, fsub2(zero, p)), fsub2(p, fsub2(y, ab))));
    float2 h = make_float2(x.ent[k], x.ent[k + 1]), v = zero;
    if (A.ref_logp) v = kl_of(fsub2(make_float2(x.ref[k], x.ref[k + 1]), logp)).kl;
    if (!x.on[k]) y.x = z.x = h.x = v.x = 0.f;
    if (!x.on[k + 1]) y.y = z.y = h.y = v.y = 0.f;
    const float2 s = fadd2(hi, y), bb = fsub2(s, hi);
    lo = fadd2(lo, fadd2(z, fadd2(fsub2(hi, fsub2(s, bb)), fsub2(y, bb))));
    hi = s;
    kl = fadd2(kl, v);
    ent = fadd2(ent, h);
    if (x.on[k]) counts += t.clipped_x ? 0x10001u : 1u;
    if (x.on[k + 1]) counts += t.clipped_y ? 0x10001u : 1u;
  }
  return Partial{add(Sum2{hi.x, lo.x}, Sum2{hi.y, lo.y}), kl.x + kl.y, ent.x + ent.y, counts};
}

// The block's record of its chunk, complete in thread 0.  The threads' sums meet in shared memory,
// where one warp per quantity adds them: trees in every warp took a third of the time.
__device__ __forceinline__ Record chunk_record(const PolicyArgs& A, const Chunk& c) {
  __shared__ float s_hi[kPolicyThreads], s_lo[kPolicyThreads], s_kl[kPolicyThreads], s_h[kPolicyThreads];
  __shared__ float s_out[2];
  __shared__ uint32_t s_counts[kPolicyThreads / 32];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const Partial mine = c.hi - c.lo == kPolicyChunk ? sum_tokens<true>(A, c) : sum_tokens<false>(A, c);
  s_hi[tid] = mine.policy.hi;
  s_lo[tid] = mine.policy.lo;
  s_kl[tid] = mine.kl;
  s_h[tid] = mine.ent;
  const uint32_t counts = __reduce_add_sync(0xffffffffu, mine.counts);
  if (lane == 0) s_counts[warp] = counts;
  __syncthreads();
  Record r{{0.f, 0.f}, 0.f, 0.f, 0u, c.seg};
  if (warp == 0) {
#pragma unroll
    for (int w = 0; w < kPolicyThreads / 32; ++w) r.policy = add(r.policy, Sum2{s_hi[32 * w + lane], s_lo[32 * w + lane]});
    r.policy = warp_sum(r.policy);
  } else if (warp <= 2) {
    const float* from = warp == 1 ? s_kl : s_h;
    float v = 0.f;
#pragma unroll
    for (int w = 0; w < kPolicyThreads / 32; ++w) v += from[32 * w + lane];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    if (lane == 0) s_out[warp - 1] = v;
  }
  __syncthreads();
  r.kl = s_out[0];
  r.ent = s_out[1];
#pragma unroll
  for (int w = 0; w < kPolicyThreads / 32; ++w) r.counts += s_counts[w];
  return r;
}

// Run by one block: live tokens per segment (integer sums, so their order does not matter),
// the segments' weights, and the weighted sums of the records in a fixed order.  Up to
// BATCH * THREADS records are held in registers between the two passes over them.
template <int THREADS, int BATCH>
__device__ __forceinline__ void finish(const PolicyArgs& A, const Record* rec, int blocks, int N, int* live) {
  __shared__ Sum2 part[3][THREADS / 32];
  __shared__ int total, beyond_bound;
  const int tid = threadIdx.x;
  Record r[BATCH];
  auto load = [&](int first) {
#pragma unroll
    for (int k = 0; k < BATCH; ++k) {
      const int b = first + k * THREADS;
      r[k].counts = 0;
      if (b < blocks) r[k] = rec[b];
    }
  };
  int sum_live = 0, sum_beyond = 0;
  for (int first = tid; first < blocks; first += BATCH * THREADS) {
    load(first);
#pragma unroll
    for (int k = 0; k < BATCH; ++k) {
      const int n = r[k].counts & 0xffff;
      if (n) atomicAdd(&live[r[k].seg], n);
      sum_live += n;
      sum_beyond += r[k].counts >> 16;
    }
  }
  if (tid == 0) total = beyond_bound = 0;
  __syncthreads();
  sum_live = __reduce_add_sync(0xffffffffu, sum_live);
  sum_beyond = __reduce_add_sync(0xffffffffu, sum_beyond);
  if ((tid & 31) == 0 && sum_live) {
    atomicAdd(&total, sum_live);
    atomicAdd(&beyond_bound, sum_beyond);
  }
  __syncthreads();
  auto weight = [&](int n) {
    if (!live[n]) return 0.f;
    return A.reduction == 0 ? 1.f / (float)total : A.reduction == 1 ? 1.f / ((float)N * (float)live[n]) : 1.f / (float)N;
  };
  for (int n = tid; n < N; n += THREADS) A.weights[n] = weight(n);
  Sum2 p{0.f, 0.f}, q = p, h = p;
  for (int first = tid; first < blocks; first += BATCH * THREADS) {
    if (blocks > BATCH * THREADS) load(first);
#pragma unroll
    for (int k = 0; k < BATCH; ++k) {
      if (!r[k].counts) continue;
      const float w = weight(r[k].seg);
      p = add(p, times(w, r[k].policy));
      q = add(q, times(w, Sum2{r[k].kl, 0.f}));
      h = add(h, times(w, Sum2{r[k].ent, 0.f}));
    }
  }
  p = warp_sum(p);
  q = warp_sum(q);
  h = warp_sum(h);
  if ((tid & 31) == 0) {
    part[0][tid >> 5] = p;
    part[1][tid >> 5] = q;
    part[2][tid >> 5] = h;
  }
  __syncthreads();
  if (tid >= 32) return;
  const bool in = tid < THREADS / 32;
  const Sum2 zero{0.f, 0.f};
  p = warp_sum(in ? part[0][tid] : zero);
  q = warp_sum(in ? part[1][tid] : zero);
  h = warp_sum(in ? part[2][tid] : zero);
  if (tid == 0) {
    const double dp = -value(p), dq = value(q), dh = value(h);
    // a term without a coefficient is a statistic alone: 0 * inf or 0 * NaN must not reach the loss
    const double kl = A.kl_coef != 0.0 ? A.kl_coef * dq : 0.0, ent = A.entropy_coef != 0.0 ? A.entropy_coef * dh : 0.0;
    A.loss[0] = (float)(dp + kl - ent);
    A.stats[0] = (float)dp;
    A.stats[1] = (float)dq;
    A.stats[2] = (float)dh;
    A.stats[3] = total ? (float)beyond_bound / (float)total : 0.f;
  }
}

template <int CAP>
__global__ void __launch_bounds__(kPolicyThreads, 6) policy_fwd_kernel(const PolicyArgs A,
                                                                    const __grid_constant__ SegTable<CAP> seg,
                                                                    const __grid_constant__ BlockIndex index) {
  const Chunk c = chunk_of(seg, index, blockIdx.x);
  const Record r = chunk_record(A, c);
  if (threadIdx.x == 0) static_cast<Record*>(A.records)[blockIdx.x] = r;
}

constexpr int kFinishThreads = 512;
// Records that a thread holds between the two passes; those of larger batches are read twice.  It hardly
// matters: 4, 8, 10 and 16 (the most without spills) took the same time within the clock's 1 us at 0.5 to 8 million
// tokens, cold, and 4 took 89 us against 87 at 12 million.
constexpr int kFinishBatch = 8;

// Starts when the blocks that make the records have exited; what comes before the wait overlaps with the rest of
// that grid's end (nothing there triggers an earlier start).
__global__ void __launch_bounds__(kFinishThreads) policy_finish_kernel(const PolicyArgs A, int blocks, int N) {
  __shared__ int live[kMaxSegs + 1];
  for (int n = threadIdx.x; n < N; n += kFinishThreads) live[n] = 0;
  __syncthreads();
  cudaGridDependencySynchronize();
  finish<kFinishThreads, kFinishBatch>(A, static_cast<const Record*>(A.records), blocks, N, live);
}

// The whole forward as one cluster of gridDim.x <= kClusterBlocks blocks.
__global__ void __launch_bounds__(kPolicyThreads, 6) policy_cluster_kernel(const PolicyArgs A,
                                                                        const __grid_constant__ SegTable<kSmallSegs> seg,
                                                                        const __grid_constant__ BlockIndex index) {
  __shared__ Record rec[kClusterBlocks];
  __shared__ int live[kClusterBlocks];  // no more segments than blocks
  cg::cluster_group cluster = cg::this_cluster();
  auto started = cluster.barrier_arrive();  // the first block has to run before its memory is written
  const Chunk c = chunk_of(seg, index, blockIdx.x);
  const Record r = chunk_record(A, c);
  cluster.barrier_wait(std::move(started));
  if (threadIdx.x == 0) {
    *cluster.map_shared_rank(&rec[blockIdx.x], 0) = r;
    if (blockIdx.x == 0)
      for (int n = 0; n < kClusterBlocks; ++n) live[n] = 0;
  }
  cluster.sync();
  if (blockIdx.x == 0) finish<kPolicyThreads, 1>(A, rec, gridDim.x, seg.N, live);
}

template <bool FULL>
__device__ __forceinline__ void token_gradients(const PolicyArgs& A, const Chunk& c) {
  Tokens x;
  load_tokens<FULL, false>(A, c, x);
  const float w = A.dloss[0] * A.weights[c.seg], wh = -(float)A.entropy_coef * w, b = (float)A.kl_coef;
  float *dlogp = A.dlogp + c.lo + threadIdx.x, *dent = A.dentropy ? A.dentropy + c.lo + threadIdx.x : nullptr;
#pragma unroll
  for (int k = 0; k < kPerThread; k += 2) {
    if (!FULL && c.lo + k * kPolicyThreads >= c.hi) break;
    const float2 logp = make_float2(x.logp[k], x.logp[k + 1]), a = make_float2(x.adv[k], x.adv[k + 1]);
    const Term t = term_of<false>(A, logp, make_float2(x.old[k], x.old[k + 1]), a);
    float2 g = fmul2(a, fadd2(t.base, fadd2(t.v, t.rest)));  // sign turned by the factor below
    if (t.clipped_x) g.x = 0.f;
    if (t.clipped_y) g.y = 0.f;
    if (A.ref_logp) g = ffma2(both(b), kl_of(fsub2(make_float2(x.ref[k], x.ref[k + 1]), logp)).slope, g);
    g = fmul2(g, both(-w));
    if (exists<FULL>(c, k)) {
      dlogp[k * kPolicyThreads] = x.on[k] ? g.x : 0.f;
      if (dent) dent[k * kPolicyThreads] = x.on[k] ? wh : 0.f;
    }
    if (exists<FULL>(c, k + 1)) {
      dlogp[(k + 1) * kPolicyThreads] = x.on[k + 1] ? g.y : 0.f;
      if (dent) dent[(k + 1) * kPolicyThreads] = x.on[k + 1] ? wh : 0.f;
    }
  }
}

template <int CAP>
__global__ void __launch_bounds__(kPolicyThreads, 6) policy_bwd_kernel(const PolicyArgs A,
                                                                       const __grid_constant__ SegTable<CAP> seg,
                                                                       const __grid_constant__ BlockIndex index) {
  const Chunk c = chunk_of(seg, index, blockIdx.x);
  if (c.hi - c.lo == kPolicyChunk) token_gradients<true>(A, c);
  else if (c.lo < c.hi) token_gradients<false>(A, c);
}

template <int CAP>
cudaError_t launch_policy_c(bool backward, const PolicyArgs& a, int N, const int32_t* off, int blocks,
                            cudaStream_t st) {
  const SegTable<CAP> s = make_segs<CAP>(0, N, off);
  const BlockIndex x = make_index(N, off, blocks);
  if (backward) {
    policy_bwd_kernel<CAP><<<blocks, kPolicyThreads, 0, st>>>(a, s, x);
    return cudaGetLastError();
  }
  cudaError_t e;
  if constexpr (CAP == kSmallSegs) {
    if (blocks <= kClusterBlocks) {
      cudaLaunchConfig_t cfg = {};
      cfg.gridDim = dim3(blocks);
      cfg.blockDim = dim3(kPolicyThreads);
      cfg.stream = st;
      cudaLaunchAttribute attr;
      attr.id = cudaLaunchAttributeClusterDimension;
      attr.val.clusterDim.x = blocks;
      attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
      cfg.attrs = &attr;
      cfg.numAttrs = 1;
      return cudaLaunchKernelEx(&cfg, policy_cluster_kernel, a, s, x);
    }
  }
  policy_fwd_kernel<CAP><<<blocks, kPolicyThreads, 0, st>>>(a, s, x);
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  return launch_behind(policy_finish_kernel, dim3(1), dim3(kFinishThreads), st, a, blocks, N);
}

int policy_blocks(int N, const int32_t* off) { return first_block(off[N], N); }

}  // namespace

cudaError_t launch_policy(bool backward, const PolicyArgs& a, int N, const int32_t* off, cudaStream_t st) {
  const int blocks = policy_blocks(N, off);
  return N <= kSmallSegs ? launch_policy_c<kSmallSegs>(backward, a, N, off, blocks, st)
                         : launch_policy_c<kMaxSegs>(backward, a, N, off, blocks, st);
}

size_t policy_workspace_bytes(int N, const int32_t* off) { return (size_t)policy_blocks(N, off) * sizeof(Record); }

}  // namespace dkv
