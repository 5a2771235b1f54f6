// rope.cu -- per-head RMS norm of q and k with the position rotation, forward and
// backward: the step that turns the projections' rows into the q and k that
// dualkv_fwd reads, and dualkv_bwd's dq and dk into the projections' gradients.
//
// For a row x of one head (D values) at position p:
//   r = (mean x^2 + eps)^-1/2,  n = x r (w + w0)         (n = x without weights)
//   y = R(p) n: the pair j < rope_dim/2 is turned by the angle p f_j
//   pairs: (j, j + rope_dim/2), or (2j, 2j + 1) when interleaved; the rest passes
// backward, with dn = R(-p) dy and u = dn (w + w0):
//   dw = sum over rows and heads of dn x r,   dx = r u - x r^3 mean(u x)
//
// Both passes read each value once and write each once (the backward recomputes
// r from x instead of loading it) and are bound by HBM bandwidth.  One warp
// takes one packed row with all its heads: the row's cosines and sines are
// computed once and stay in registers while the warp walks the heads.  A head
// is spread over G = D/16 lanes; a lane holds two 16-byte vectors A and B
// chosen so that both members of every pair lie in the same lane.
//
// Angles: p f is formed in fp64, reduced to turns there, and only the fraction
// of a turn goes to fp32; at p = 10^5 a product in fp32 would already be off by
// 0.004 rad.  Everything else is fp32; the only rounding to bf16 is the final
// one.  Weight gradients are summed in fp32 per warp, then per block and across
// blocks in a fixed order.
#include <cuda_bf16.h>

#include "kernels.h"
#include "segs.cuh"

namespace dkv {

namespace {

constexpr int kRopeWarps = 8;
constexpr int kRopeThreads = kRopeWarps * 32;

__device__ __forceinline__ void unpack8(const uint4& v, float* f) {
  const __nv_bfloat162* h = reinterpret_cast<const __nv_bfloat162*>(&v);
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const float2 t = __bfloat1622float2(h[e]);
    f[2 * e] = t.x;
    f[2 * e + 1] = t.y;
  }
}

__device__ __forceinline__ uint4 pack8(const float* f) {
  uint4 v;
  __nv_bfloat162* h = reinterpret_cast<__nv_bfloat162*>(&v);
#pragma unroll
  for (int e = 0; e < 4; ++e) h[e] = __floats2bfloat162_rn(f[2 * e], f[2 * e + 1]);
  return v;
}

// Where a lane's vectors A and B lie in a head, and whether they are turned.
struct LaneMap {
  int a, b;   // element offsets
  bool turn;
};

template <int D>
__device__ __forceinline__ LaneMap lane_map(int i, int half, bool inter) {
  if (inter) return LaneMap{16 * i, 16 * i + 8, 8 * i < half};
  if (8 * i < half) return LaneMap{8 * i, half + 8 * i, true};
  return LaneMap{16 * i, 16 * i + 8, false};  // 2 half + 16 (i - half / 8)
}

// cos and sin of the 8 angles of this lane's pairs (1 and 0 in lanes that are not
// turned).  The S = 32/G lanes with the same i share the work.
template <int D>
__device__ __forceinline__ void row_angles(int p, const float* __restrict__ inv_freq, int i, int slot, bool turn,
                                           float* cs, float* sn) {
  constexpr int G = D / 16, S = 32 / G, PER = 8 / S;
  float c[PER], s[PER];
#pragma unroll
  for (int e = 0; e < PER; ++e) {
    c[e] = 1.f;
    s[e] = 0.f;
    if (turn) {
      double t = (double)p * (double)__ldg(inv_freq + 8 * i + slot * PER + e) * 0.15915494309189533577;
      t -= rint(t);
      sincospif((float)(2.0 * t), &s[e], &c[e]);
    }
  }
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    cs[e] = __shfl_sync(0xffffffffu, c[e % PER], (e / PER) * G + i);
    sn[e] = __shfl_sync(0xffffffffu, s[e % PER], (e / PER) * G + i);
  }
}

// Turns the pairs of (a, b) by the angles (cs, sn).
__device__ __forceinline__ void rotate(float* a, float* b, const float* cs, const float* sn, bool inter, float sign) {
  if (inter) {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float c0 = cs[e], s0 = sign * sn[e], c1 = cs[4 + e], s1 = sign * sn[4 + e];
      const float x0 = a[2 * e], x1 = a[2 * e + 1], z0 = b[2 * e], z1 = b[2 * e + 1];
      a[2 * e] = x0 * c0 - x1 * s0;
      a[2 * e + 1] = x1 * c0 + x0 * s0;
      b[2 * e] = z0 * c1 - z1 * s1;
      b[2 * e + 1] = z1 * c1 + z0 * s1;
    }
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float s = sign * sn[e], x = a[e], z = b[e];
      a[e] = x * cs[e] - z * s;
      b[e] = z * cs[e] + x * s;
    }
  }
}

template <int G>
__device__ __forceinline__ float group_sum(float v) {
#pragma unroll
  for (int o = G / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// The lane's 16 effective weights w + w0.
__device__ __forceinline__ void load_weights(const void* w, int f32, float w0, const LaneMap& m, float* wa, float* wb) {
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    wa[e] = w0 + (f32 ? __ldg(static_cast<const float*>(w) + m.a + e)
                      : __bfloat162float(static_cast<const __nv_bfloat16*>(w)[m.a + e]));
    wb[e] = w0 + (f32 ? __ldg(static_cast<const float*>(w) + m.b + e)
                      : __bfloat162float(static_cast<const __nv_bfloat16*>(w)[m.b + e]));
  }
}

template <int D>
__device__ __forceinline__ void fwd_heads(const RopeArgs& A, const __nv_bfloat16* __restrict__ x,
                                          __nv_bfloat16* __restrict__ y, int H, const LaneMap& m, int slot,
                                          const void* w, const float* cs, const float* sn) {
  constexpr int G = D / 16, S = 32 / G;
  float wa[8], wb[8];
  if (w) load_weights(w, A.weight_f32, A.w0, m, wa, wb);
  for (int h0 = 0; h0 < H; h0 += S) {
    const int h = h0 + slot;
    float a[8], b[8];
    uint4 va = make_uint4(0, 0, 0, 0), vb = va;
    if (h < H) {
      va = __ldg(reinterpret_cast<const uint4*>(x + h * D + m.a));
      vb = __ldg(reinterpret_cast<const uint4*>(x + h * D + m.b));
    }
    unpack8(va, a);
    unpack8(vb, b);
    if (w) {
      float ss = 0.f;
#pragma unroll
      for (int e = 0; e < 8; ++e) ss += a[e] * a[e] + b[e] * b[e];
      const float r = rsqrtf(group_sum<G>(ss) * (1.f / D) + A.eps);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        a[e] *= r * wa[e];
        b[e] *= r * wb[e];
      }
    }
    rotate(a, b, cs, sn, A.inter, 1.f);
    if (h < H) {
      *reinterpret_cast<uint4*>(y + h * D + m.a) = pack8(a);
      *reinterpret_cast<uint4*>(y + h * D + m.b) = pack8(b);
    }
  }
}

template <int D, int CAP>
__global__ void __launch_bounds__(kRopeThreads) rope_fwd_kernel(const RopeArgs A,
                                                                const __grid_constant__ SegTable<CAP> seg) {
  constexpr int G = D / 16;
  const int lane = threadIdx.x & 31, slot = lane / G, i = lane % G;
  const LaneMap m = lane_map<D>(i, A.half, A.inter);
  for (int64_t t = (int64_t)blockIdx.x * kRopeWarps + (threadIdx.x >> 5); t < A.T; t += (int64_t)gridDim.x * kRopeWarps) {
    float cs[8], sn[8];
    row_angles<D>(position_of(seg, (int)t), A.inv_freq, i, slot, m.turn, cs, sn);
    fwd_heads<D>(A, A.q + t * A.q_stride, A.q_out + t * A.q_out_stride, A.Hq, m, slot, A.q_weight, cs, sn);
    fwd_heads<D>(A, A.k + t * A.k_stride, A.k_out + t * A.k_out_stride, A.Hkv, m, slot, A.k_weight, cs, sn);
  }
}

// Input gradients of one row's heads; adds the lane's weight gradients to (da, db).
template <int D>
__device__ __forceinline__ void bwd_heads(const RopeArgs& A, const __nv_bfloat16* __restrict__ x,
                                          const __nv_bfloat16* __restrict__ dy, __nv_bfloat16* __restrict__ dx, int H,
                                          const LaneMap& m, int slot, const void* w, const float* cs, const float* sn,
                                          float* da, float* db) {
  constexpr int G = D / 16, S = 32 / G;
  float wa[8], wb[8];
  if (w) load_weights(w, A.weight_f32, A.w0, m, wa, wb);
  for (int h0 = 0; h0 < H; h0 += S) {
    const int h = h0 + slot;
    uint4 va = make_uint4(0, 0, 0, 0), vb = va, ga = va, gb = va;
    if (h < H) {
      ga = __ldg(reinterpret_cast<const uint4*>(dy + h * D + m.a));
      gb = __ldg(reinterpret_cast<const uint4*>(dy + h * D + m.b));
      if (w) {
        va = __ldg(reinterpret_cast<const uint4*>(x + h * D + m.a));
        vb = __ldg(reinterpret_cast<const uint4*>(x + h * D + m.b));
      }
    }
    float g[8], f[8];
    unpack8(ga, g);
    unpack8(gb, f);
    rotate(g, f, cs, sn, A.inter, -1.f);
    if (w) {
      float a[8], b[8];
      unpack8(va, a);
      unpack8(vb, b);
      float ss = 0.f, ux = 0.f;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        ss += a[e] * a[e] + b[e] * b[e];
        ux += g[e] * wa[e] * a[e] + f[e] * wb[e] * b[e];
      }
      const float r = rsqrtf(group_sum<G>(ss) * (1.f / D) + A.eps);
      const float mean = group_sum<G>(ux) * r * (1.f / D);  // mean(u x r)
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float xa = a[e] * r, xb = b[e] * r;
        da[e] += g[e] * xa;
        db[e] += f[e] * xb;
        g[e] = r * (g[e] * wa[e] - xa * mean);
        f[e] = r * (f[e] * wb[e] - xb * mean);
      }
    }
    if (h < H) {
      *reinterpret_cast<uint4*>(dx + h * D + m.a) = pack8(g);
      *reinterpret_cast<uint4*>(dx + h * D + m.b) = pack8(f);
    }
  }
}

// Sum of the block's weight gradients in a fixed order -> out[D].
template <int D>
__device__ __forceinline__ void block_weight_grad(float* smem, const LaneMap& m, int slot, const float* da,
                                                  const float* db, float* out) {
  constexpr int G = D / 16, S = 32 / G;
  const int warp = threadIdx.x >> 5;
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    float a = da[e], b = db[e];
#pragma unroll
    for (int o = G; o < 32; o <<= 1) {
      a += __shfl_xor_sync(0xffffffffu, a, o);
      b += __shfl_xor_sync(0xffffffffu, b, o);
    }
    if (slot == 0) {
      smem[warp * D + m.a + e] = a;
      smem[warp * D + m.b + e] = b;
    }
  }
  __syncthreads();
  for (int d = threadIdx.x; d < D; d += kRopeThreads) {
    float v = 0.f;
#pragma unroll
    for (int k = 0; k < kRopeWarps; ++k) v += smem[k * D + d];
    out[d] = v;
  }
  __syncthreads();
}

template <int D, int CAP>
__global__ void __launch_bounds__(kRopeThreads) rope_bwd_kernel(const RopeArgs A,
                                                                const __grid_constant__ SegTable<CAP> seg) {
  constexpr int G = D / 16;
  __shared__ float smem[kRopeWarps * D];
  const int lane = threadIdx.x & 31, slot = lane / G, i = lane % G;
  const LaneMap m = lane_map<D>(i, A.half, A.inter);
  float qa[8] = {}, qb[8] = {}, ka[8] = {}, kb[8] = {};
  for (int64_t t = (int64_t)blockIdx.x * kRopeWarps + (threadIdx.x >> 5); t < A.T; t += (int64_t)gridDim.x * kRopeWarps) {
    float cs[8], sn[8];
    row_angles<D>(position_of(seg, (int)t), A.inv_freq, i, slot, m.turn, cs, sn);
    bwd_heads<D>(A, A.q + t * A.q_stride, A.dq_out + t * A.Hq * D, A.q_out + t * A.q_out_stride, A.Hq, m, slot,
                 A.q_weight, cs, sn, qa, qb);
    bwd_heads<D>(A, A.k + t * A.k_stride, A.dk_out + t * A.Hkv * D, A.k_out + t * A.k_out_stride, A.Hkv, m, slot,
                 A.k_weight, cs, sn, ka, kb);
  }
  if (A.q_weight) {
    block_weight_grad<D>(smem, m, slot, qa, qb, A.partial + (int64_t)blockIdx.x * 2 * D);
    block_weight_grad<D>(smem, m, slot, ka, kb, A.partial + (int64_t)blockIdx.x * 2 * D + D);
  }
}

// Weight gradients: column d of the blocks' partial sums, added in block order.
// A block of 32 x 8 threads takes 32 columns; the 8 rows of threads take
// contiguous eighths of the blocks, which are then added in order.
__global__ void __launch_bounds__(256) rope_weight_kernel(const float* __restrict__ partial, int blocks, int D,
                                                          float* __restrict__ dqw, float* __restrict__ dkw) {
  __shared__ double part[8][32];
  const int col = blockIdx.x * 32 + threadIdx.x, per = (blocks + 7) / 8;
  const int b0 = threadIdx.y * per, b1 = min(blocks, b0 + per);
  double v = 0.0;
#pragma unroll 4
  for (int b = b0; b < b1; ++b) v += (double)partial[(int64_t)b * 2 * D + col];
  part[threadIdx.y][threadIdx.x] = v;
  __syncthreads();
  if (threadIdx.y) return;
  for (int k = 1; k < 8; ++k) v += part[k][threadIdx.x];
  if (col < D) dqw[col] = (float)v;
  else dkw[col - D] = (float)v;
}

template <int D>
cudaError_t launch_rope_d(bool backward, const RopeArgs& a, int P, int N, const int32_t* off, int grid,
                          cudaStream_t st) {
  if (N <= kSmallSegs) {
    const SegTable<kSmallSegs> s = make_segs<kSmallSegs>(P, N, off);
    if (backward) rope_bwd_kernel<D, kSmallSegs><<<grid, kRopeThreads, 0, st>>>(a, s);
    else rope_fwd_kernel<D, kSmallSegs><<<grid, kRopeThreads, 0, st>>>(a, s);
  } else {
    const SegTable<kMaxSegs> s = make_segs<kMaxSegs>(P, N, off);
    if (backward) rope_bwd_kernel<D, kMaxSegs><<<grid, kRopeThreads, 0, st>>>(a, s);
    else rope_fwd_kernel<D, kMaxSegs><<<grid, kRopeThreads, 0, st>>>(a, s);
  }
  return cudaGetLastError();
}

int rope_grid(int64_t T) {
  const int64_t need = (T + kRopeWarps - 1) / kRopeWarps;
  return (int)(need < kRopeMaxBlocks ? need : kRopeMaxBlocks);
}

}  // namespace

cudaError_t launch_rope(bool backward, int D, const RopeArgs& a, int P, int N, const int32_t* off, float* dqw,
                        float* dkw, cudaStream_t st) {
  const int grid = rope_grid(a.T);
  cudaError_t e;
  switch (D) {
    case 64:
      e = launch_rope_d<64>(backward, a, P, N, off, grid, st);
      break;
    case 128:
      e = launch_rope_d<128>(backward, a, P, N, off, grid, st);
      break;
    case 512:
      e = launch_rope_d<512>(backward, a, P, N, off, grid, st);
      break;
    default:
      return cudaErrorInvalidValue;
  }
  if (e != cudaSuccess || !backward || !a.q_weight) return e;
  rope_weight_kernel<<<2 * D / 32, dim3(32, 8), 0, st>>>(a.partial, grid, D, dqw, dkw);
  return cudaGetLastError();
}

size_t rope_workspace_bytes(int64_t T, int D) { return (size_t)rope_grid(T) * 2 * D * sizeof(float); }

}  // namespace dkv
