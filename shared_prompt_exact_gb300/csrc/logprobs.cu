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
// each gradient once.  Both are bound by HBM bandwidth.  Statistics are fp32.
#include <cuda_bf16.h>
#include <math_constants.h>

#include "kernels.h"
#include "ptx.cuh"
#include "segs.cuh"

namespace dkv {

namespace {

constexpr int kLogpThreads = 512;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ float to_f(float x) { return x; }
__device__ __forceinline__ float to_f(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ void from_f(float x, float* d) { *d = x; }
__device__ __forceinline__ void from_f(float x, __nv_bfloat16* d) { *d = __float2bfloat16_rn(x); }

__device__ __forceinline__ void unpack(const uint4& v, float (&f)[4]) {
  f[0] = __uint_as_float(v.x);
  f[1] = __uint_as_float(v.y);
  f[2] = __uint_as_float(v.z);
  f[3] = __uint_as_float(v.w);
}
__device__ __forceinline__ void unpack(const uint4& v, float (&f)[8]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    f[2 * e] = __uint_as_float(w[e] << 16);
    f[2 * e + 1] = __uint_as_float(w[e] & 0xffff0000u);
  }
}
__device__ __forceinline__ uint4 pack(const float (&f)[4]) {
  return make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3]));
}
__device__ __forceinline__ uint4 pack(const float (&f)[8]) {
  uint4 v;
  __nv_bfloat162* h = reinterpret_cast<__nv_bfloat162*>(&v);
#pragma unroll
  for (int e = 0; e < 4; ++e) h[e] = __floats2bfloat162_rn(f[2 * e], f[2 * e + 1]);
  return v;
}

// A row's 16-byte vectors: elements [head, head + nv * E), between two ragged ends.
template <typename T>
struct RowVectors {
  static constexpr int E = 16 / sizeof(T);
  int head, nv, tail;  // tail: first element behind the vectors
  __device__ __forceinline__ RowVectors(const T* row, int V) {
    head = (int)(((16 - (reinterpret_cast<uintptr_t>(row) & 15)) & 15) / sizeof(T));
    head = head < V ? head : V;
    nv = (V - head) / E;
    tail = head + nv * E;
  }
};

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
// where c = scale log2(e).  While only -inf has been seen m is -inf and s, t are 0 (NaN after a NaN).
struct Running {
  float m, s, t;
};

// (z - m) c, with 0 in place of a maximum of -inf.
__device__ __forceinline__ float floor_of(float m) { return m == -CUDART_INF_F ? 0.f : m; }

// Moves (s, t) from their maximum to a larger one.
__device__ __forceinline__ void rebase(Running& r, float m, float c) {
  if (r.m != -CUDART_INF_F) {
    const float d = (r.m - floor_of(m)) * c, f = ex2(d);
    // d is -inf only below a maximum of +inf, whose own term makes the sums NaN
    r.t = (r.t + d * r.s) * f;
    r.s *= f;
  }
  r.m = m;
}

__device__ __forceinline__ Running join(Running a, Running b, float c) {
  const float m = fmaxf(a.m, b.m);
  rebase(a, m, c);
  rebase(b, m, c);
  return Running{m, a.s + b.s, a.t + b.t};
}

template <bool ENT, int K>
__device__ __forceinline__ void absorb(Running& r, const float (&z)[K], float c) {
  float m = z[0];
#pragma unroll
  for (int e = 1; e < K; ++e) m = fmaxf(m, z[e]);
  if (m > r.m) rebase(r, m, c);
  const float base = floor_of(r.m);
#pragma unroll
  for (int e = 0; e < K; ++e) {
    const float y = (z[e] - base) * c, x = ex2(y);
    r.s += x;
    if (ENT) r.t = fmaf(x, fmaxf(y, -1e30f), r.t);  // a masked logit adds 0, not 0 * inf
  }
}

__device__ __forceinline__ Running block_join(Running r, float c) {
  __shared__ Running part[kLogpThreads / 32];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const Running b{__shfl_xor_sync(0xffffffffu, r.m, o), __shfl_xor_sync(0xffffffffu, r.s, o),
                    __shfl_xor_sync(0xffffffffu, r.t, o)};
    r = join(r, b, c);
  }
  if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = r;
  __syncthreads();
  r = part[0];
  for (int k = 1; k < kLogpThreads / 32; ++k) r = join(r, part[k], c);
  return r;
}

template <typename T, bool ENT, int CAP>
__global__ void __launch_bounds__(kLogpThreads) logp_fwd_kernel(const LogpArgs A,
                                                                const __grid_constant__ SegTable<CAP> seg) {
  constexpr int E = RowVectors<T>::E;
  const int64_t row = blockIdx.x;
  const int n = seg.off[seg.N], tid = threadIdx.x;
  const bool shared_row = seg.P > 0 && row == 0;
  int open = -1, mine = -1, live = 0;
  if (shared_row) {
    for (int s = tid; s < seg.N; s += kLogpThreads)
      if (seg.off[s] < seg.off[s + 1] && token_at(A, seg.off[s]) >= 0) live = 1;
    live = __syncthreads_or(live);
  } else {
    mine = predicted(seg, row, &open);
    if (mine >= 0) live = token_at(A, mine) >= 0;
    if (seg.P == 0 && row == 0 && tid == 0 && n > 0) {  // token 0 opens its segment
      A.logp[0] = 0.f;
      if (ENT) A.entropy[0] = 0.f;
    }
  }
  const float c = A.scale * kLog2e;
  const T* x = static_cast<const T*>(A.logits) + row * A.stride;
  if (live) {
    const RowVectors<T> v(x, A.V);
    Running r{-CUDART_INF_F, 0.f, 0.f};
    const uint4* xv = reinterpret_cast<const uint4*>(x + v.head);
    for (int k = tid; k < v.nv; k += kLogpThreads) {
      float z[E];
      unpack(__ldg(xv + k), z);
      absorb<ENT>(r, z, c);
    }
    for (int k = tid; k < v.head + A.V - v.tail; k += kLogpThreads) {
      const float z[1] = {to_f(x[k < v.head ? k : v.tail + k - v.head])};
      absorb<ENT>(r, z, c);
    }
    r = block_join(r, c);
    // r.s is 0 only in a row that is -inf throughout: lse and logp are -inf there, H is 0
    const bool none = r.s == 0.f;
    const float ln_sum = logf(r.s), ent = none ? 0.f : ln_sum - r.t / r.s * kLn2;
    auto write = [&](int i) {
      const int tok = token_at(A, i);
      // smaller terms than z - lse, so a likelier token keeps more digits
      const float lp = tok < 0 ? 0.f : none ? -CUDART_INF_F : (to_f(x[tok]) - r.m) * A.scale - ln_sum;
      A.logp[i] = lp;
      if (ENT) A.entropy[i] = tok < 0 ? 0.f : ent;
    };
    if (shared_row) {
      for (int s = tid; s < seg.N; s += kLogpThreads)
        if (seg.off[s] < seg.off[s + 1]) write(seg.off[s]);
    } else if (tid == 0) {
      write(mine);
    }
    if (tid == 0 && A.lse) A.lse[row] = none ? -CUDART_INF_F : fmaf(r.m, A.scale, ln_sum);
    return;
  }
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

// Gradient of one logit z (raw): p (k0 + k1 d), d = z scale - lse.  d is formed before the
// scaling to base 2, so that its rounding is relative to d and not to z.
template <bool ENT>
__device__ __forceinline__ float grad_of(float z, float scale, float lse, float k0, float k1) {
  const float d = fmaf(z, scale, -lse), p = ex2(d * kLog2e);
  return ENT ? p * fmaf(fmaxf(d, -1e30f), k1, k0) : p * k0;
}

template <typename T, bool ENT, int CAP>
__global__ void __launch_bounds__(kLogpThreads) logp_bwd_kernel(const LogpArgs A,
                                                                const __grid_constant__ SegTable<CAP> seg) {
  constexpr int E = RowVectors<T>::E;
  extern __shared__ uint32_t dyn[];
  int* s_tok = reinterpret_cast<int*>(dyn);              // [N] the shared row's targets (-1: none)
  float* s_g = reinterpret_cast<float*>(dyn) + seg.N;    // [N] their upstream gradients
  float* s_v = s_g + seg.N;                              // [N] the targets' logit gradients
  const int64_t row = blockIdx.x;
  const int tid = threadIdx.x;
  const bool shared_row = seg.P > 0 && row == 0;
  const T* x = static_cast<const T*>(A.logits) + row * A.stride;
  T* y = static_cast<T*>(A.dlogits) + row * A.dstride;
  const float lse = A.lse[row];
  float g = 0.f, h = 0.f, ent = 0.f;
  int tok = -1;
  if (shared_row) {
    int any = -1;
    for (int s = tid; s < seg.N; s += kLogpThreads) {
      const int i = seg.off[s];
      const int t = i < seg.off[s + 1] ? token_at(A, i) : -1;
      s_tok[s] = t;
      s_g[s] = t >= 0 ? A.dlogp[i] : 0.f;
      if (t >= 0) {
        g += A.dlogp[i];
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
  } else {
    int open;
    const int i = predicted(seg, row, &open);
    if (i >= 0) tok = token_at(A, i);
    if (tok >= 0) {
      g = A.dlogp[i];
      if (ENT) {
        h = A.dentropy[i];
        ent = A.entropy[i];
      }
    }
  }
  const RowVectors<T> v(y, A.V);
  const int ends = v.head + A.V - v.tail;
  uint4* yv = reinterpret_cast<uint4*>(y + v.head);
  bool targets = false;  // a shared row whose gradients cancel in g may still have targets
  if (shared_row) {
    for (int s = tid; s < seg.N; s += kLogpThreads) targets |= s_g[s] != 0.f;
    targets = __syncthreads_or(targets);
  }
  if ((g == 0.f && h == 0.f && !targets) || lse == -CUDART_INF_F) {
    // nothing flows into this row (or it is masked throughout): zeros, without reading it
    for (int k = tid; k < v.nv; k += kLogpThreads) yv[k] = make_uint4(0, 0, 0, 0);
    for (int k = tid; k < ends; k += kLogpThreads) from_f(0.f, y + (k < v.head ? k : v.tail + k - v.head));
    return;
  }
  const float scale = A.scale;
  const float k1 = -scale * h, k0 = -scale * fmaf(h, ent, g);
  // The targets' gradients, from logits that an in-place pass is about to overwrite.  Equal
  // targets of the shared row all get the same sum over them, in segment order.
  float vt = 0.f;
  if (shared_row) {
    for (int s = tid; s < seg.N; s += kLogpThreads) {
      const int t = s_tok[s];
      if (t < 0) continue;
      float sum = 0.f;
      for (int u = 0; u < seg.N; ++u) sum += s_tok[u] == t ? s_g[u] : 0.f;
      s_v[s] = fmaf(scale, sum, grad_of<ENT>(to_f(x[t]), scale, lse, k0, k1));
    }
  } else if (tid == 0) {
    vt = fmaf(scale, g, grad_of<ENT>(to_f(x[tok]), scale, lse, k0, k1));
  }
  __syncthreads();
  if (((reinterpret_cast<uintptr_t>(x) ^ reinterpret_cast<uintptr_t>(y)) & 15) == 0) {
    const uint4* xv = reinterpret_cast<const uint4*>(x + v.head);
    for (int k = tid; k < v.nv; k += kLogpThreads) {
      float z[E];
      unpack(xv[k], z);
#pragma unroll
      for (int e = 0; e < E; ++e) z[e] = grad_of<ENT>(z[e], scale, lse, k0, k1);
      yv[k] = pack(z);
    }
    for (int k = tid; k < ends; k += kLogpThreads) {
      const int j = k < v.head ? k : v.tail + k - v.head;
      from_f(grad_of<ENT>(to_f(x[j]), scale, lse, k0, k1), y + j);
    }
  } else {
    for (int j = tid; j < A.V; j += kLogpThreads) from_f(grad_of<ENT>(to_f(x[j]), scale, lse, k0, k1), y + j);
  }
  __syncthreads();
  if (shared_row) {
    for (int s = tid; s < seg.N; s += kLogpThreads)
      if (s_tok[s] >= 0) from_f(s_v[s], y + s_tok[s]);
  } else if (tid == 0) {
    from_f(vt, y + tok);
  }
}

template <typename T, bool ENT, int CAP>
cudaError_t launch_logp_c(bool backward, const LogpArgs& a, int P, int N, const int32_t* off, cudaStream_t st) {
  const SegTable<CAP> s = make_segs<CAP>(P, N, off);
  const unsigned grid = (unsigned)(off[N] + (P > 0 ? 1 : 0));
  if (!backward) {
    logp_fwd_kernel<T, ENT, CAP><<<grid, kLogpThreads, 0, st>>>(a, s);
    return cudaGetLastError();
  }
  const size_t smem = (size_t)N * 12;
  if (smem > 32768) {  // beyond 48 KB with the kernel's static arrays
    const cudaError_t e = cudaFuncSetAttribute(logp_bwd_kernel<T, ENT, CAP>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               kMaxSegs * 12);
    if (e != cudaSuccess) return e;
  }
  logp_bwd_kernel<T, ENT, CAP><<<grid, kLogpThreads, smem, st>>>(a, s);
  return cudaGetLastError();
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
