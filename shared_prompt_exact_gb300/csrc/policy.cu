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
// A block takes up to kPolicyChunk tokens of ONE segment and writes one record of sums;
// a second, single block turns the records into weights and the loss.  Blocks are
// numbered without a list: segment n owns blocks [off[n] / chunk + n, off[n + 1] / chunk + n + 1),
// at least as many as it has chunks.  Sums are fp32 over a thread's tokens and fp64
// from there on, in a fixed order.  Up to about a million tokens launch latency
// is all the time; beyond that HBM bandwidth.
#include <cuda_runtime.h>

#include "kernels.h"
#include "segs.cuh"

namespace dkv {

namespace {

constexpr int kPolicyThreads = 256;

struct Record {
  double policy, kl, ent;
  int clipped, live, seg, pad;
};

// The block's segment and its token range [lo, hi) (empty when the segment needs fewer blocks).
struct Chunk {
  int seg, lo, hi;
};
template <int CAP>
__device__ __forceinline__ Chunk chunk_of(const SegTable<CAP>& s, int block) {
  int lo = 0, hi = s.N - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (s.off[mid] / kPolicyChunk + mid <= block) lo = mid;
    else hi = mid - 1;
  }
  const int c = block - (s.off[lo] / kPolicyChunk + lo);
  const int64_t begin = (int64_t)s.off[lo] + (int64_t)c * kPolicyChunk;
  const int end = s.off[lo + 1];
  if (begin >= end) return Chunk{lo, end, end};
  return Chunk{lo, (int)begin, (int)(begin + kPolicyChunk < end ? begin + kPolicyChunk : end)};
}

// a - b as the rounded difference and what rounding took away (0 where the difference is not finite).
__device__ __forceinline__ float exact_diff(float a, float b, float* err) {
  const float d = a - b, bb = d - a;
  const float e = (a - (d - bb)) - (b + bb);
  *err = fabsf(d) <= 3.4e38f ? e : 0.f;
  return d;
}
__device__ __forceinline__ bool above(float d, float e, const Bound& t) { return d > t.hi || (d == t.hi && e > t.lo); }
__device__ __forceinline__ bool below(float d, float e, const Bound& t) { return d < t.hi || (d == t.hi && e < t.lo); }

// e^x - x - 1: its series where the difference would cancel.
__device__ __forceinline__ float kl_of(float x) {
  if (fabsf(x) >= 0.5f) return expm1f(x) - x;
  float p = 1.f / 362880.f;
  p = fmaf(p, x, 1.f / 40320.f);
  p = fmaf(p, x, 1.f / 5040.f);
  p = fmaf(p, x, 1.f / 720.f);
  p = fmaf(p, x, 1.f / 120.f);
  p = fmaf(p, x, 1.f / 24.f);
  p = fmaf(p, x, 1.f / 6.f);
  p = fmaf(p, x, 0.5f);
  return p * x * x;
}

struct Term {
  float ratio, bounded;
  bool clipped;
};
__device__ __forceinline__ Term term_of(const PolicyArgs& A, float logp, float old, float adv) {
  Term t;
  float e;
  const float d = exact_diff(logp, old, &e);
  t.ratio = expf(d);
  if (fabsf(d) < 80.f) t.ratio = fmaf(t.ratio, e, t.ratio);
  t.bounded = t.ratio;
  t.clipped = false;
  if (adv > 0.f) {
    if (above(d, e, A.up)) {
      t.bounded = A.ratio_up;
      t.clipped = true;
    }
  } else if (adv < 0.f) {
    if (below(d, e, A.down)) {
      t.bounded = A.ratio_down;
      t.clipped = true;
    } else if (A.has_dual && above(d, e, A.dual)) {
      t.bounded = A.ratio_dual;
      t.clipped = true;
    }
  } else if (adv == 0.f) {
    t.ratio = t.bounded = 0.f;  // not 0 * inf
  }
  return t;
}

__device__ __forceinline__ double block_sum(double v, double* part) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = v;
  __syncthreads();
  v = 0.0;
  for (int k = 0; k < (int)blockDim.x / 32; ++k) v += part[k];
  return v;
}

template <int CAP>
__global__ void __launch_bounds__(kPolicyThreads) policy_fwd_kernel(const PolicyArgs A,
                                                                    const __grid_constant__ SegTable<CAP> seg) {
  __shared__ double part[kPolicyThreads / 32];
  const Chunk c = chunk_of(seg, blockIdx.x);
  float policy = 0.f, kl = 0.f, ent = 0.f;
  int clipped = 0, live = 0;
  for (int i = c.lo + threadIdx.x; i < c.hi; i += kPolicyThreads) {
    if (A.mask && !A.mask[i]) continue;
    const float logp = A.logp[i], adv = A.adv[A.per_token ? i : c.seg];
    const Term t = term_of(A, logp, A.old_logp[i], adv);
    policy -= adv * t.bounded;
    clipped += t.clipped;
    ++live;
    if (A.ref_logp) kl += kl_of(A.ref_logp[i] - logp);
    if (A.entropy) ent += A.entropy[i];
  }
  const double sp = block_sum((double)policy, part), sk = block_sum((double)kl, part), se = block_sum((double)ent, part);
  const int nc = (int)block_sum((double)clipped, part), nl = (int)block_sum((double)live, part);
  if (threadIdx.x == 0) static_cast<Record*>(A.records)[blockIdx.x] = Record{sp, sk, se, nc, nl, c.seg, 0};
}

constexpr int kFinishThreads = 1024;

// One block: live tokens per segment (integer sums, so their order does not matter), the
// segments' weights, and the weighted sums of the records in a fixed order.
__global__ void __launch_bounds__(kFinishThreads) policy_finish_kernel(const PolicyArgs A, int blocks, int N) {
  __shared__ int live[kMaxSegs + 1];
  __shared__ double part[kFinishThreads / 32];
  __shared__ int total;
  const Record* rec = static_cast<const Record*>(A.records);
  for (int n = threadIdx.x; n < N; n += kFinishThreads) live[n] = 0;
  if (threadIdx.x == 0) total = 0;
  __syncthreads();
  int clipped = 0;
  for (int b = threadIdx.x; b < blocks; b += kFinishThreads) {
    if (!rec[b].live) continue;
    atomicAdd(&live[rec[b].seg], rec[b].live);
    atomicAdd(&total, rec[b].live);
    clipped += rec[b].clipped;
  }
  __syncthreads();
  auto weight = [&](int n) {
    if (!live[n]) return 0.0;
    return A.reduction == 0 ? 1.0 / total : A.reduction == 1 ? 1.0 / ((double)N * live[n]) : 1.0 / N;
  };
  for (int n = threadIdx.x; n < N; n += kFinishThreads) A.weights[n] = (float)weight(n);
  double p = 0.0, k = 0.0, e = 0.0;
  for (int b = threadIdx.x; b < blocks; b += kFinishThreads) {
    if (!rec[b].live) continue;
    const double w = weight(rec[b].seg);
    p += w * rec[b].policy;
    k += w * rec[b].kl;
    e += w * rec[b].ent;
  }
  p = block_sum(p, part);
  k = block_sum(k, part);
  e = block_sum(e, part);
  const double nc = block_sum((double)clipped, part);
  if (threadIdx.x == 0) {
    A.loss[0] = (float)(p + A.kl_coef * k - A.entropy_coef * e);
    A.stats[0] = (float)p;
    A.stats[1] = (float)k;
    A.stats[2] = (float)e;
    A.stats[3] = total ? (float)(nc / total) : 0.f;
  }
}

template <int CAP>
__global__ void __launch_bounds__(kPolicyThreads) policy_bwd_kernel(const PolicyArgs A,
                                                                    const __grid_constant__ SegTable<CAP> seg) {
  const Chunk c = chunk_of(seg, blockIdx.x);
  if (c.lo >= c.hi) return;
  const double w = (double)A.dloss[0] * (double)A.weights[c.seg];
  const float wf = (float)w, wh = (float)(-A.entropy_coef * w), b = (float)A.kl_coef;
  for (int i = c.lo + threadIdx.x; i < c.hi; i += kPolicyThreads) {
    const bool on = !A.mask || A.mask[i];
    float g = 0.f;
    if (on) {
      const float logp = A.logp[i], adv = A.adv[A.per_token ? i : c.seg];
      const Term t = term_of(A, logp, A.old_logp[i], adv);
      g = t.clipped ? 0.f : -adv * t.ratio;
      if (A.ref_logp) g = fmaf(-b, expm1f(A.ref_logp[i] - logp), g);
      g *= wf;
    }
    A.dlogp[i] = g;
    if (A.dentropy) A.dentropy[i] = on ? wh : 0.f;
  }
}

template <int CAP>
cudaError_t launch_policy_c(bool backward, const PolicyArgs& a, int N, const int32_t* off, int blocks,
                            cudaStream_t st) {
  const SegTable<CAP> s = make_segs<CAP>(0, N, off);
  if (backward) {
    policy_bwd_kernel<CAP><<<blocks, kPolicyThreads, 0, st>>>(a, s);
    return cudaGetLastError();
  }
  policy_fwd_kernel<CAP><<<blocks, kPolicyThreads, 0, st>>>(a, s);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  policy_finish_kernel<<<1, kFinishThreads, 0, st>>>(a, blocks, N);
  return cudaGetLastError();
}

int policy_blocks(int N, const int32_t* off) { return off[N] / kPolicyChunk + N; }

}  // namespace

cudaError_t launch_policy(bool backward, const PolicyArgs& a, int N, const int32_t* off, cudaStream_t st) {
  const int blocks = policy_blocks(N, off);
  return N <= kSmallSegs ? launch_policy_c<kSmallSegs>(backward, a, N, off, blocks, st)
                         : launch_policy_c<kMaxSegs>(backward, a, N, off, blocks, st);
}

size_t policy_workspace_bytes(int N, const int32_t* off) { return (size_t)policy_blocks(N, off) * sizeof(Record); }

}  // namespace dkv
