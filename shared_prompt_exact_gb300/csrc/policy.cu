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
// A block takes up to kPolicyChunk tokens of ONE segment, all of whose loads are issued before
// the first is used, and makes one record of sums (fp32 trees); a single block then turns the
// records into weights and the loss, with compensated fp32 sums (two values each) in a fixed
// order.  fp64 adds run at two lanes per clock and SM here: with them in the trees a call on 4M
// tokens took 172 us instead of 32.  Blocks are numbered without a list: segment n owns blocks
// [off[n] / chunk + n, off[n + 1] / chunk + n + 1), at least as many as it has chunks.  Up to
// kClusterBlocks blocks run as one cluster whose first block joins the records from its shared
// memory; more write them to the workspace for a second launch.
//
// Up to some 100,000 tokens a call is launch latency (about 6 us in a graph).  At 4.04M tokens
// (1,024 responses, every input in use) the forward takes 32 us, 2.7 TB/s: 26 for the records,
// bound by memory latency and issue together (about 160 instructions a token and warp), the rest
// the join; the gradients take 24 us, 4.2 TB/s.  Chunks of 1,024 and 4 tokens a thread beat 2,048
// and 8 (40 against 50 us cold): more resident threads outweigh fewer loads in flight each.
#include <cooperative_groups.h>
#include <cuda_runtime.h>

#include "kernels.h"
#include "segs.cuh"

namespace dkv {

namespace {

namespace cg = cooperative_groups;

constexpr int kPolicyThreads = 256;
constexpr int kPerThread = kPolicyChunk / kPolicyThreads;
constexpr int kClusterBlocks = 8;

// A chunk's sums; counts holds the live tokens and, in the upper half, those beyond a bound.
struct alignas(16) Record {
  float policy, kl, ent;
  uint32_t counts;
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

// a - b as the rounded difference and what rounding took away (finite even where the difference is not).
__device__ __forceinline__ float exact_diff(float a, float b, float* err) {
  const float d = a - b, bb = d - a;
  const float e = (a - (d - bb)) - (b + bb);
  *err = fmaxf(e, -1e30f);  // not NaN
  return d;
}
// The sign of (d + e) - t: d - t.hi is exact where the two are close, and elsewhere larger than the rest.
__device__ __forceinline__ float beyond(float d, float e, const Bound& t) { return (d - t.hi) + (e - t.lo); }

// e^x - x - 1 and e^x - 1: by the series of the former below |x| = 1, where differences would cancel.
struct Kl {
  float kl, slope;
};
__device__ __forceinline__ Kl kl_of(float x) {
  if (!(fabsf(x) < 1.f)) {
    const float q = expf(x) - 1.f;
    return Kl{q - x, q};
  }
  float p = 1.f / 39916800.f;
  p = fmaf(p, x, 1.f / 3628800.f);
  p = fmaf(p, x, 1.f / 362880.f);
  p = fmaf(p, x, 1.f / 40320.f);
  p = fmaf(p, x, 1.f / 5040.f);
  p = fmaf(p, x, 1.f / 720.f);
  p = fmaf(p, x, 1.f / 120.f);
  p = fmaf(p, x, 1.f / 24.f);
  p = fmaf(p, x, 1.f / 6.f);
  p = fmaf(p, x, 0.5f) * x * x;
  return Kl{p, p + x};
}

// A token's ratio, the ratio that its policy term uses, and whether that is a bound.
struct Term {
  float ratio, bounded;
  bool clipped;
};
__device__ __forceinline__ Term term_of(const PolicyArgs& A, float logp, float old, float adv) {
  float e;
  const float d = exact_diff(logp, old, &e);
  float ratio = expf(d);
  const bool gain = adv > 0.f, loss = adv < 0.f;
  const float x = beyond(d, e, Bound{gain ? A.up.hi : A.down.hi, gain ? A.up.lo : A.down.lo});
  Term t;
  t.clipped = gain ? x > 0.f : loss && x < 0.f;
  t.bounded = t.clipped ? (gain ? A.ratio_up : A.ratio_down) : ratio;
  if (A.has_dual && loss && beyond(d, e, A.dual) > 0.f) {
    t.clipped = true;
    t.bounded = A.ratio_dual;
  }
  if (adv == 0.f) ratio = t.bounded = 0.f;  // not 0 * inf
  t.ratio = ratio;
  return t;
}

// A thread's tokens of a chunk: lo + tid + k * threads.  Masked ones are loaded, not used.
struct Tokens {
  float logp[kPerThread], old[kPerThread], adv[kPerThread], ref[kPerThread], ent[kPerThread];
  bool in[kPerThread], on[kPerThread];
};
template <bool ENT>
__device__ __forceinline__ void load_tokens(const PolicyArgs& A, const Chunk& c, Tokens& t) {
  const int64_t at = (int64_t)c.lo + threadIdx.x;
  const int left = c.hi - c.lo - (int)threadIdx.x;
  const float *logp = A.logp + at, *old = A.old_logp + at, *ref = A.ref_logp + at, *ent = A.entropy + at;
  const float* adv = A.per_token ? A.adv + at : A.adv + c.seg;
  const uint8_t* mask = A.mask + at;
  const bool per_token = A.per_token, has_ref = A.ref_logp, has_ent = ENT && A.entropy, has_mask = A.mask;
#pragma unroll
  for (int k = 0; k < kPerThread; ++k) {
    t.in[k] = t.on[k] = k * kPolicyThreads < left;
    t.logp[k] = t.old[k] = t.adv[k] = t.ref[k] = t.ent[k] = 0.f;
    if (t.in[k]) {
      t.logp[k] = logp[k * kPolicyThreads];
      t.old[k] = old[k * kPolicyThreads];
      t.adv[k] = adv[per_token ? k * kPolicyThreads : 0];
      if (has_ref) t.ref[k] = ref[k * kPolicyThreads];
      if (has_ent) t.ent[k] = ent[k * kPolicyThreads];
      if (has_mask) t.on[k] = mask[k * kPolicyThreads] != 0;
    }
  }
}

// A sum kept as hi + lo, with the rounding errors of the additions in lo.
struct Sum2 {
  float hi, lo;
};
__device__ __forceinline__ Sum2 add(const Sum2& a, const Sum2& b) {
  const float s = a.hi + b.hi, bb = s - a.hi;
  const float e = (a.hi - (s - bb)) + (b.hi - bb) + a.lo + b.lo;
  return Sum2{s, fabsf(s) <= 3.4e38f ? e : 0.f};
}
__device__ __forceinline__ Sum2 warp_sum(Sum2 v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1)
    v = add(v, Sum2{__shfl_xor_sync(0xffffffffu, v.hi, o), __shfl_xor_sync(0xffffffffu, v.lo, o)});
  return v;
}
__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// The block's record of its chunk, complete in thread 0.
__device__ __forceinline__ Record chunk_record(const PolicyArgs& A, const Chunk& c) {
  __shared__ Record part[kPolicyThreads / 32];
  const int tid = threadIdx.x;
  Tokens x;
  load_tokens<true>(A, c, x);
  float policy = 0.f, kl = 0.f, h = 0.f;
  uint32_t counts = 0;
#pragma unroll
  for (int k = 0; k < kPerThread; ++k) {
    if (c.lo + k * kPolicyThreads >= c.hi) break;  // the same for the whole block
    const Term t = term_of(A, x.logp[k], x.old[k], x.adv[k]);
    if (x.on[k]) {
      policy = fmaf(-x.adv[k], t.bounded, policy);
      h += x.ent[k];
      counts += t.clipped ? 0x10001u : 1u;
    }
    if (A.ref_logp) {
      const float v = kl_of(x.ref[k] - x.logp[k]).kl;
      if (x.on[k]) kl += v;
    }
  }
  Record r{warp_sum(policy), warp_sum(kl), warp_sum(h), __reduce_add_sync(0xffffffffu, counts)};
  if ((tid & 31) == 0) part[tid >> 5] = r;
  __syncthreads();
  if (tid == 0) {
#pragma unroll
    for (int w = 1; w < kPolicyThreads / 32; ++w) {
      r.policy += part[w].policy;
      r.kl += part[w].kl;
      r.ent += part[w].ent;
      r.counts += part[w].counts;
    }
  }
  return r;
}

// Run by one block: live tokens per segment (integer sums, so their order does not matter),
// the segments' weights, and the weighted sums of the records in a fixed order.  Up to
// BATCH * THREADS records are held in registers between the two passes over them.
template <int THREADS, int BATCH>
__device__ __forceinline__ void finish(const PolicyArgs& A, const Record* rec, const int* segs, int blocks, int N,
                                       int* live) {
  __shared__ Sum2 part[3][THREADS / 32];
  __shared__ int total, beyond_bound;
  const int tid = threadIdx.x;
  Record r[BATCH];
  int seg[BATCH];
  auto load = [&](int first) {
#pragma unroll
    for (int k = 0; k < BATCH; ++k) {
      const int b = first + k * THREADS;
      r[k] = Record{0.f, 0.f, 0.f, 0u};
      seg[k] = 0;
      if (b < blocks) {
        r[k] = rec[b];
        seg[k] = segs[b];
      }
    }
  };
  int sum_live = 0, sum_beyond = 0;
  for (int first = tid; first < blocks; first += BATCH * THREADS) {
    load(first);
#pragma unroll
    for (int k = 0; k < BATCH; ++k) {
      const int n = r[k].counts & 0xffff;
      if (n) atomicAdd(&live[seg[k]], n);
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
      const float w = weight(seg[k]);
      p = add(p, Sum2{w * r[k].policy, 0.f});
      q = add(q, Sum2{w * r[k].kl, 0.f});
      h = add(h, Sum2{w * r[k].ent, 0.f});
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
    const double dp = (double)p.hi + p.lo, dq = (double)q.hi + q.lo, dh = (double)h.hi + h.lo;
    A.loss[0] = (float)(dp + A.kl_coef * dq - A.entropy_coef * dh);
    A.stats[0] = (float)dp;
    A.stats[1] = (float)dq;
    A.stats[2] = (float)dh;
    A.stats[3] = total ? (float)beyond_bound / (float)total : 0.f;
  }
}

// The workspace: the records of `blocks` blocks, then their segments.
__device__ __forceinline__ int* segs_of(const PolicyArgs& A, int blocks) {
  return reinterpret_cast<int*>(static_cast<Record*>(A.records) + blocks);
}

template <int CAP>
__global__ void __launch_bounds__(kPolicyThreads, 6) policy_fwd_kernel(const PolicyArgs A,
                                                                    const __grid_constant__ SegTable<CAP> seg,
                                                                    const __grid_constant__ BlockIndex index) {
  const Chunk c = chunk_of(seg, index, blockIdx.x);
  const Record r = chunk_record(A, c);
  if (threadIdx.x == 0) {
    static_cast<Record*>(A.records)[blockIdx.x] = r;
    segs_of(A, gridDim.x)[blockIdx.x] = c.seg;
  }
}

constexpr int kFinishThreads = 1024;

// Launched while the records are still being made: everything before the wait overlaps with that.
__global__ void __launch_bounds__(kFinishThreads) policy_finish_kernel(const PolicyArgs A, int blocks, int N) {
  __shared__ int live[kMaxSegs + 1];
  for (int n = threadIdx.x; n < N; n += kFinishThreads) live[n] = 0;
  __syncthreads();
  cudaGridDependencySynchronize();
  finish<kFinishThreads, 6>(A, static_cast<const Record*>(A.records), segs_of(A, blocks), blocks, N, live);
}

// The whole forward as one cluster of gridDim.x <= kClusterBlocks blocks.
__global__ void __launch_bounds__(kPolicyThreads, 6) policy_cluster_kernel(const PolicyArgs A,
                                                                        const __grid_constant__ SegTable<kSmallSegs> seg,
                                                                        const __grid_constant__ BlockIndex index) {
  __shared__ Record rec[kClusterBlocks];
  __shared__ int segs[kClusterBlocks], live[kClusterBlocks];  // no more segments than blocks
  cg::cluster_group cluster = cg::this_cluster();
  const Chunk c = chunk_of(seg, index, blockIdx.x);
  const Record r = chunk_record(A, c);
  if (threadIdx.x == 0) {
    *cluster.map_shared_rank(&rec[blockIdx.x], 0) = r;
    *cluster.map_shared_rank(&segs[blockIdx.x], 0) = c.seg;
    if (blockIdx.x == 0)
      for (int n = 0; n < kClusterBlocks; ++n) live[n] = 0;
  }
  cluster.sync();
  if (blockIdx.x == 0) finish<kPolicyThreads, 1>(A, rec, segs, gridDim.x, seg.N, live);
}

template <int CAP>
__global__ void __launch_bounds__(kPolicyThreads, 6) policy_bwd_kernel(const PolicyArgs A,
                                                                    const __grid_constant__ SegTable<CAP> seg,
                                                                    const __grid_constant__ BlockIndex index) {
  const Chunk c = chunk_of(seg, index, blockIdx.x);
  if (c.lo >= c.hi) return;
  Tokens x;
  load_tokens<false>(A, c, x);
  const float w = A.dloss[0] * A.weights[c.seg], wh = -(float)A.entropy_coef * w, b = (float)A.kl_coef;
  float *dlogp = A.dlogp + c.lo + threadIdx.x, *dent = A.dentropy ? A.dentropy + c.lo + threadIdx.x : nullptr;
#pragma unroll
  for (int k = 0; k < kPerThread; ++k) {
    if (c.lo + k * kPolicyThreads >= c.hi) break;
    const Term t = term_of(A, x.logp[k], x.old[k], x.adv[k]);
    float g = t.clipped ? 0.f : -x.adv[k] * t.ratio;
    if (A.ref_logp) g = fmaf(-b, kl_of(x.ref[k] - x.logp[k]).slope, g);
    if (x.in[k]) {
      dlogp[k * kPolicyThreads] = x.on[k] ? g * w : 0.f;
      if (dent) dent[k * kPolicyThreads] = x.on[k] ? wh : 0.f;
    }
  }
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
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(1);
  cfg.blockDim = dim3(kFinishThreads);
  cfg.stream = st;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, policy_finish_kernel, a, blocks, N);
}

int policy_blocks(int N, const int32_t* off) { return first_block(off[N], N); }

}  // namespace

cudaError_t launch_policy(bool backward, const PolicyArgs& a, int N, const int32_t* off, cudaStream_t st) {
  const int blocks = policy_blocks(N, off);
  return N <= kSmallSegs ? launch_policy_c<kSmallSegs>(backward, a, N, off, blocks, st)
                         : launch_policy_c<kMaxSegs>(backward, a, N, off, blocks, st);
}

size_t policy_workspace_bytes(int N, const int32_t* off) { return (size_t)policy_blocks(N, off) * (sizeof(Record) + sizeof(int)); }

}  // namespace dkv
