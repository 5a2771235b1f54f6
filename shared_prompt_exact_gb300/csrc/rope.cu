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
// takes one packed row with all its heads, so the row's cosines and sines are
// computed once and stay in registers; a head is spread over G = D/16 lanes, a
// lane holding two 16-byte vectors A and B chosen so that both members of every
// pair lie in it.  Loads run ahead of their use through shared memory
// (cp.async); arithmetic is on f32x2 pairs, because with plain fp32 the backward
// was bound by issue (64 % of the slots) as much as by memory.  Measured: forward
// 222 us for 71,680 rows of 32 + 8 heads of 128 (6.6 TB/s, 0.97 of the measured
// copy bandwidth; 331 us with loads straight into registers), backward 393 us for
// 84,997 such rows (6.7 TB/s; 868 us) and 180 us for 36,522 rows of 8 + 2 heads of
// 512 (6.2 TB/s; 496 us, with loads of every other vector).
//
// Angles: p f is formed in 64-bit fixed point as a fraction of a turn, and only
// that fraction goes to fp32; at p = 10^5 a product in fp32 would already be off
// by 0.004 rad.  Everything else is fp32; the only rounding to bf16 is the final
// one.  Weight gradients are summed in fp32 per lane, per block and across blocks, in
// a fixed order.
#include <cuda_bf16.h>

#include "kernels.h"
#include "launch.cuh"
#include "ptx.cuh"
#include "rope.cuh"
#include "segs.cuh"

namespace dkv {

namespace {

constexpr int kRopeWarps = 8;
constexpr int kRopeThreads = kRopeWarps * 32;
// Steps in a lane's ring: the one in use and those that its copies run ahead.  Three keep 32 KB
// (forward) and 64 KB (backward) per SM in flight; with 4 to 6 and grids of 608 to 2432 blocks the
// times above moved by less than 4 % (304 blocks: 7 % more).  Two blocks per SM: three leave the backward 80 registers, and
// it then spills (464 us instead of 404).
constexpr int kDepth = 3;

// What a block keeps in shared memory: frequencies, effective weights w + w0 of q and k (split_at),
// and every warp's cosines and sines.
template <int D>
struct RopeShared {
  alignas(16) float w[2][D];
  alignas(16) float cs[kRopeWarps][D / 2];
  alignas(16) float sn[kRopeWarps][D / 2];
  uint64_t freq[D / 2];
};

template <int D>
__device__ __forceinline__ void load_shared(const RopeArgs& A, RopeShared<D>& s) {
  for (int j = threadIdx.x; j < A.half; j += kRopeThreads) s.freq[j] = turn_fraction(A.inv_freq[j]);
  if (A.q_weight) {
    for (int d = threadIdx.x; d < 2 * D; d += kRopeThreads) {
      const void* w = d < D ? A.q_weight : A.k_weight;
      const int e = d % D;
      s.w[d / D][split_at(e, D)] = A.w0 + (A.weight_f32 ? static_cast<const float*>(w)[e]
                                                    : __bfloat162float(static_cast<const __nv_bfloat16*>(w)[e]));
    }
  }
  __syncthreads();
}

// A warp's walk: rows t, t + stride, ..., in each row the steps [begin, end) of those that take q's
// heads, S = 32 / G at a time, and those behind them that take k's.  Block rows (blockIdx.y) share a
// row's steps: the first `qparts` of them q's and the others k's, or (`both`) all of them all steps.
template <int D>
struct Walk {
  static constexpr int S = 32 / (D / 16);
  int nq, begin, end;
  int64_t first, stride;
  __device__ __forceinline__ Walk(const RopeArgs& A, int qparts, bool both, int warp) {
    nq = (A.Hq + S - 1) / S;
    const int nk = (A.Hkv + S - 1) / S, y = (int)blockIdx.y, kparts = (int)gridDim.y - qparts;
    if (both) {
      begin = (nq + nk) * y / (int)gridDim.y;
      end = (nq + nk) * (y + 1) / (int)gridDim.y;
    } else {
      begin = y < qparts ? nq * y / qparts : nq + nk * (y - qparts) / kparts;
      end = y < qparts ? nq * (y + 1) / qparts : nq + nk * (y + 1 - qparts) / kparts;
    }
    first = (int64_t)blockIdx.x * kRopeWarps + warp;
    stride = (int64_t)gridDim.x * kRopeWarps;
  }
};

// The copies' place in the walk.  x and g are the lane's vector A in the head and in its upstream
// gradient (backward); vector B lies m.b - m.a behind.
template <int D, bool BWD>
struct Ahead {
  static constexpr int S = Walk<D>::S;
  const __nv_bfloat16 *x, *g;
  int h, H, s;
  int64_t t;

  __device__ __forceinline__ void place(const RopeArgs& A, const Walk<D>& w, int slot, int a) {
    const bool is_q = s < w.nq;
    h = slot + (s - (is_q ? 0 : w.nq)) * S;
    H = is_q ? A.Hq : A.Hkv;
    x = (is_q ? A.q + t * A.q_stride : A.k + t * A.k_stride) + h * D + a;
    if (BWD) g = (is_q ? A.dq_out : A.dk_out) + (t * H + h) * D + a;
  }
  __device__ __forceinline__ void start(const RopeArgs& A, const Walk<D>& w, int slot, int a) {
    t = w.first;
    s = w.begin;
    place(A, w, slot, a);
  }
  __device__ __forceinline__ void step(const RopeArgs& A, const Walk<D>& w, int slot, int a) {
    h += S;
    x += S * D;
    if (BWD) g += S * D;
    ++s;
    if (s != w.nq && s != w.end) return;
    if (s == w.end) {
      t += w.stride;
      s = w.begin;
    }
    place(A, w, slot, a);
  }
};

template <int D, int CAP>
__global__ void __launch_bounds__(kRopeThreads, 2) rope_fwd_kernel(const RopeArgs A,
                                                                    const __grid_constant__ SegTable<CAP> seg) {
  constexpr int G = D / 16, S = 32 / G;
  extern __shared__ uint4 ring[];  // [kDepth][2][threads]
  __shared__ RopeShared<D> sh;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, slot = lane / G, i = lane % G;
  const LaneMap m = lane_map<D>(i, A.half, A.inter);
  const bool norm = A.q_weight != nullptr;
  const int db = m.b - m.a;
  const Walk<D> walk(A, 0, true, warp);
  uint4* mine = ring + threadIdx.x;
  Ahead<D, false> ahead;
  ahead.start(A, walk, slot, m.a);
  auto fetch = [&](int stage) {
    if (ahead.t < A.T) {
      uint4* to = mine + 2 * stage * kRopeThreads;
      if (ahead.h < ahead.H) {
        copy16(to, ahead.x);
        copy16(to + kRopeThreads, ahead.x + db);
      }
      ahead.step(A, walk, slot, m.a);
    }
    copies_commit();
  };
#pragma unroll
  for (int k = 0; k < kDepth - 1; ++k) fetch(k);
  load_shared<D>(A, sh);
  int stage = 0;
  for (int64_t t = walk.first; t < A.T; t += walk.stride) {
    const Angles ang =
        row_angles(position_of(seg, (int)t), sh.freq, A.half, sh.cs[warp], sh.sn[warp], lane, m, A.inter);
    auto heads = [&](int from, int to, int H, const float* w, __nv_bfloat16* y) {
      y += from * S * D;
      for (int s = from, h = slot + from * S; s < to; ++s, h += S, y += S * D) {
        fetch(stage == 0 ? kDepth - 1 : stage - 1);
        copies_wait<kDepth - 1>();
        Vec8 a = unpack8(mine[2 * stage * kRopeThreads]), b = unpack8(mine[(2 * stage + 1) * kRopeThreads]);
        stage = stage == kDepth - 1 ? 0 : stage + 1;
        if (norm) {
          float2 ss = make_float2(0.f, 0.f);
#pragma unroll
          for (int e = 0; e < 4; ++e) ss = ffma2(b.v[e], b.v[e], ffma2(a.v[e], a.v[e], ss));
          const float r = rsqrtf(group_sum<G>(ss) * (1.f / D) + A.eps);
          const float2 rr = make_float2(r, r);
          const Vec8 wa = load8(w + m.a / 2, w + D / 2 + m.a / 2), wb = load8(w + m.b / 2, w + D / 2 + m.b / 2);
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            a.v[e] = fmul2(a.v[e], fmul2(rr, wa.v[e]));
            b.v[e] = fmul2(b.v[e], fmul2(rr, wb.v[e]));
          }
        }
        rotate(a, b, ang.cs, ang.sn, ang.neg, A.inter);
        if (h < H) {
          *reinterpret_cast<uint4*>(y) = pack8(a);
          *reinterpret_cast<uint4*>(y + db) = pack8(b);
        }
      }
    };
    heads(walk.begin, min(walk.end, walk.nq), A.Hq, sh.w[0], A.q_out + t * A.q_out_stride + slot * D + m.a);
    heads(max(walk.begin - walk.nq, 0), walk.end - walk.nq, A.Hkv, sh.w[1],
          A.k_out + t * A.k_out_stride + slot * D + m.a);
  }
}

// One head's input gradient from the gradient turned back (g, f) and the head (a, b), in place; adds
// the lane's weight gradients to (da, db).  `head`: whether the lane's slot has a head in this step; one
// without adds nothing (its zeros alone would not see to that: with eps = 0 their norm is 0 * inf).
template <int D>
__device__ __forceinline__ void norm_backward(Vec8& g, Vec8& f, const Vec8& a, const Vec8& b, const float* w,
                                              const LaneMap& m, float eps, bool head, Vec8& da, Vec8& db) {
  constexpr int G = D / 16;
  const Vec8 wa = load8(w + m.a / 2, w + D / 2 + m.a / 2), wb = load8(w + m.b / 2, w + D / 2 + m.b / 2);
  float2 ss = make_float2(0.f, 0.f), ux = ss;
  Vec8 ua, ub;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    ua.v[e] = fmul2(g.v[e], wa.v[e]);
    ub.v[e] = fmul2(f.v[e], wb.v[e]);
    ss = ffma2(b.v[e], b.v[e], ffma2(a.v[e], a.v[e], ss));
    ux = ffma2(ub.v[e], b.v[e], ffma2(ua.v[e], a.v[e], ux));
  }
  const float mean = group_sum<G>(ss) * (1.f / D) + eps, r = head ? rsqrtf(mean) : 0.f;
  const float k = -group_sum<G>(ux) * (1.f / D) * r * r * r;  // dx = r u - x r^3 mean(u x)
  const float2 rr = make_float2(r, r), kk = make_float2(k, k);
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    da.v[e] = ffma2(g.v[e], fmul2(a.v[e], rr), da.v[e]);
    db.v[e] = ffma2(f.v[e], fmul2(b.v[e], rr), db.v[e]);
    g.v[e] = ffma2(a.v[e], kk, fmul2(ua.v[e], rr));
    f.v[e] = ffma2(b.v[e], kk, fmul2(ub.v[e], rr));
  }
}

// Sum of the block's weight gradients in a fixed order -> out[D].
template <int D>
__device__ __forceinline__ void block_weight_grad(float* smem, const LaneMap& m, int slot, const Vec8& da,
                                                  const Vec8& db, float* out) {
  constexpr int G = D / 16;
  const int warp = threadIdx.x >> 5;
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const int k = vec8_at(e) >> 1;
    float a = vec8_at(e) & 1 ? da.v[k].y : da.v[k].x, b = vec8_at(e) & 1 ? db.v[k].y : db.v[k].x;
#pragma unroll
    for (int o = G; o < 32; o <<= 1) {
      a += __shfl_xor_sync(0xffffffffu, a, o);
      b += __shfl_xor_sync(0xffffffffu, b, o);
    }
    if (slot == 0) {  // value e of every vector together: neighbouring lanes write neighbouring words
      smem[warp * D + e * (D / 8) + m.a / 8] = a;
      smem[warp * D + e * (D / 8) + m.b / 8] = b;
    }
  }
  __syncthreads();
  for (int d = threadIdx.x; d < D; d += kRopeThreads) {
    float v = 0.f;
#pragma unroll
    for (int k = 0; k < kRopeWarps; ++k) v += smem[k * D + d];
    out[d % (D / 8) * 8 + d / (D / 8)] = v;
  }
  __syncthreads();
}

template <int D, int CAP>
__global__ void __launch_bounds__(kRopeThreads, 2) rope_bwd_kernel(const RopeArgs A, int qparts,
                                                                    const __grid_constant__ SegTable<CAP> seg) {
  constexpr int G = D / 16, S = 32 / G;
  extern __shared__ uint4 ring[];  // [kDepth][4][threads]
  __shared__ RopeShared<D> sh;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, slot = lane / G, i = lane % G;
  const LaneMap m = lane_map<D>(i, A.half, A.inter);
  const bool norm = A.q_weight != nullptr, is_q = (int)blockIdx.y < qparts;
  const int db = m.b - m.a;
  const Walk<D> walk(A, qparts, false, warp);
  uint4* mine = ring + threadIdx.x;
  Ahead<D, true> ahead;
  ahead.start(A, walk, slot, m.a);
  auto fetch = [&](int stage) {
    if (ahead.t < A.T) {
      uint4* to = mine + 4 * stage * kRopeThreads;
      if (ahead.h < ahead.H) {
        copy16(to, ahead.g);
        copy16(to + kRopeThreads, ahead.g + db);
        if (norm) {
          copy16(to + 2 * kRopeThreads, ahead.x);
          copy16(to + 3 * kRopeThreads, ahead.x + db);
        }
      } else {  // an idle slot's gradient is 0
#pragma unroll
        for (int v = 0; v < 4; ++v) to[v * kRopeThreads] = make_uint4(0, 0, 0, 0);
      }
      ahead.step(A, walk, slot, m.a);
    }
    copies_commit();
  };
#pragma unroll
  for (int k = 0; k < kDepth - 1; ++k) fetch(k);
  load_shared<D>(A, sh);
  Vec8 da{}, db_{};
  int stage = 0;
  const int from = walk.begin - (is_q ? 0 : walk.nq), to = walk.end - (is_q ? 0 : walk.nq), H = is_q ? A.Hq : A.Hkv;
  const float* w = sh.w[!is_q];
  __nv_bfloat16* out = (is_q ? A.q_out : A.k_out) + (from * S + slot) * D + m.a;
  const int64_t out_stride = is_q ? A.q_out_stride : A.k_out_stride;
  for (int64_t t = walk.first; t < A.T; t += walk.stride) {
    const Angles ang =
        row_angles(position_of(seg, (int)t), sh.freq, A.half, sh.cs[warp], sh.sn[warp], lane, m, A.inter);
    __nv_bfloat16* y = out + t * out_stride;
    for (int s = from; s < to; ++s) {
      fetch(stage == 0 ? kDepth - 1 : stage - 1);
      copies_wait<kDepth - 1>();
      const uint4* in = mine + 4 * stage * kRopeThreads;
      stage = stage == kDepth - 1 ? 0 : stage + 1;
      const bool head = s * S + slot < H;
      Vec8 g = unpack8(in[0]), f = unpack8(in[kRopeThreads]);
      rotate(g, f, ang.cs, ang.neg, ang.sn, A.inter);  // by minus the angle
      if (norm)
        norm_backward<D>(g, f, unpack8(in[2 * kRopeThreads]), unpack8(in[3 * kRopeThreads]), w, m, A.eps, head, da, db_);
      if (head) {
        *reinterpret_cast<uint4*>(y) = pack8(g);
        *reinterpret_cast<uint4*>(y + db) = pack8(f);
      }
      y += S * D;
    }
  }
  if (norm) {
    // every lane has waited for its own copies; the ring becomes the place of the block's sums
    copies_wait<0>();
    __syncthreads();
    block_weight_grad<D>(reinterpret_cast<float*>(ring), m, slot, da, db_,
                         A.partial + ((int64_t)blockIdx.y * gridDim.x + blockIdx.x) * D);
  }
}

// Weight gradients: column d of the blocks' partial sums, added in block order.
// A block of 32 x 32 threads takes 32 columns of q's or k's; its rows of threads take
// contiguous shares of the blocks, which are then added in order.  It may start before `partial` is
// complete, so that is not __restrict__.
__global__ void __launch_bounds__(1024) rope_weight_kernel(const float* partial, int qblocks, int kblocks, int D,
                                                           float* dqw, float* dkw) {
  __shared__ float part[32][33];
  const int c = blockIdx.x * 32 + threadIdx.x, col = c % D;
  const bool is_q = c < D;
  const int blocks = is_q ? qblocks : kblocks, per = (blocks + 31) / 32;
  const int b0 = threadIdx.y * per, b1 = min(blocks, b0 + per);
  if (!is_q) partial += (int64_t)qblocks * D;
  float v = 0.f;
  cudaGridDependencySynchronize();
#pragma unroll 8
  for (int b = b0; b < b1; ++b) v += partial[(int64_t)b * D + col];
  part[threadIdx.y][threadIdx.x] = v;
  __syncthreads();
  if (threadIdx.y) return;
#pragma unroll
  for (int k = 1; k < 32; ++k) v += part[k][threadIdx.x];
  (is_q ? dqw : dkw)[col] = v;
}

// Blocks over the rows (x) and over the steps of a row (y): as many block rows as it takes to give
// the resident warps work when rows are few (192 rows of 32 + 8 heads of 128: the backward takes 8 us
// in a graph, 10.4 with a warp walking all 10 steps of its row).  In the backward the first qparts of
// them take q's heads and the others k's, so that a lane sums one tensor's weight gradients and
// needs 16 registers less for them (410 against 422 us at 84,997 rows).
constexpr int kRopeResident = 152 * 2;
// Most blocks over the rows: 912 for the backward, whose blocks end with a sum (1,824: the same time),
// 1,824 for the forward (912: 1 % more).
constexpr int kRopeFwdBlocks = 152 * 12, kRopeBwdBlocks = 152 * 6;
struct RopeGrid {
  dim3 grid;
  int qparts;
};
RopeGrid rope_grid(bool backward, int64_t T, int Hq, int Hkv, int D) {
  const int64_t need = (T + kRopeWarps - 1) / kRopeWarps;
  const int S = 512 / D, nq = (Hq + S - 1) / S, nk = (Hkv + S - 1) / S;
  int64_t spare = kRopeResident / need;
  if (spare < 1) spare = 1;
  const int most = backward ? kRopeBwdBlocks : kRopeFwdBlocks;
  RopeGrid g;
  g.grid = dim3((unsigned)(need < most ? need : most));
  if (!backward) {
    g.qparts = 0;
    g.grid.y = (unsigned)(spare < nq + nk ? spare : nq + nk);
  } else {
    g.qparts = (int)(spare < nq ? spare : nq);
    g.grid.y = (unsigned)(g.qparts + (spare < nk ? spare : nk));
  }
  return g;
}

template <int D, int CAP>
cudaError_t launch_rope_c(bool backward, const RopeArgs& a, int P, int N, const int32_t* off, const RopeGrid& g,
                          cudaStream_t st) {
  const SegTable<CAP> s = make_segs<CAP>(P, N, off);
  const int smem = (backward ? 4 : 2) * kDepth * kRopeThreads * (int)sizeof(uint4);
  if (backward) {  // the forward stays within the 48 KB that need no asking
    const cudaError_t e = cudaFuncSetAttribute(rope_bwd_kernel<D, CAP>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
  }
  if (backward) rope_bwd_kernel<D, CAP><<<g.grid, kRopeThreads, smem, st>>>(a, g.qparts, s);
  else rope_fwd_kernel<D, CAP><<<g.grid, kRopeThreads, smem, st>>>(a, s);
  return cudaGetLastError();
}

template <int D>
cudaError_t launch_rope_d(bool backward, const RopeArgs& a, int P, int N, const int32_t* off, const RopeGrid& g,
                          cudaStream_t st) {
  return N <= kSmallSegs ? launch_rope_c<D, kSmallSegs>(backward, a, P, N, off, g, st)
                         : launch_rope_c<D, kMaxSegs>(backward, a, P, N, off, g, st);
}

}  // namespace

cudaError_t launch_rope(bool backward, int D, const RopeArgs& a, int P, int N, const int32_t* off, float* dqw,
                        float* dkw, cudaStream_t st) {
  const RopeGrid g = rope_grid(backward, a.T, a.Hq, a.Hkv, D);
  cudaError_t e;
  switch (D) {
    case 64:
      e = launch_rope_d<64>(backward, a, P, N, off, g, st);
      break;
    case 128:
      e = launch_rope_d<128>(backward, a, P, N, off, g, st);
      break;
    case 512:
      e = launch_rope_d<512>(backward, a, P, N, off, g, st);
      break;
    default:
      return cudaErrorInvalidValue;
  }
  if (e != cudaSuccess || !backward || !a.q_weight) return e;
  const int qblocks = (int)(g.grid.x * g.qparts), kblocks = (int)(g.grid.x * g.grid.y) - qblocks;
  return launch_behind(rope_weight_kernel, dim3(2 * D / 32), dim3(32, 32), st, a.partial, qblocks, kblocks, D, dqw, dkw);
}

size_t rope_workspace_bytes(int64_t T, int Hq, int Hkv, int D) {
  const dim3 grid = rope_grid(true, T, Hq, Hkv, D).grid;
  return (size_t)grid.x * grid.y * D * sizeof(float);
}

}  // namespace dkv
