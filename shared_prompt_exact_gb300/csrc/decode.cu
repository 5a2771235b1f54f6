// decode.cu -- attention of one new token per response over the paged cache.
//
// For response b of group g (prompt of P tokens, own n = lens[b] >= 0 tokens, query at P + n - 1):
//   x_k = scale q k over the tokens of the prompt and the response within the window
//   m = max x, l = sum exp(x - m), out = sum exp(x - m) v / l, lse = m + log l
// A block takes one response and head; its warps walk the keys with a running maximum, a lane
// holding D / 32 values of the head, and join their sums at the end.
#include <cuda_bf16.h>

#include "cache.cuh"
#include "kernels.h"
#include "ptx.cuh"
#include "segs.cuh"

namespace dkv {

namespace {

constexpr int kWarps = 4;

// Value d of a row of a pool.
__device__ __forceinline__ float value_at(const void* pool, const __nv_bfloat16* scales, int64_t row, int D, int d) {
  if (!scales) return __bfloat162float(static_cast<const __nv_bfloat16*>(pool)[row * D + d]);
  const uint8_t c = static_cast<const uint8_t*>(pool)[row * (D / 2) + d / 2];
  return __bfloat162float(scales[row * (D / kGroup) + d / kGroup]) * (float)((d & 1 ? c >> 4 : c & 15) - 8);
}

template <int D, int CAP>
__global__ void __launch_bounds__(kWarps * 32) decode_kernel(const DecodeArgs A, const __grid_constant__ SegTable<CAP> seg) {
  constexpr int E = D / 32;
  const int b = blockIdx.x, h = blockIdx.y, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int g = seg_of(seg, b), kvh = h / (A.Hq / A.kv.Hkv), n = A.lens[b];
  const int P = A.prompt_lens && n >= 0 ? max(0, A.prompt_lens[g]) : 0;
  const int lo = A.window > 0 ? max(0, P - A.window + n) : 0, end = P + max(n, 0);
  float q[E], o[E], m = -INFINITY, l = 0.f;
#pragma unroll
  for (int e = 0; e < E; ++e) {
    q[e] = __bfloat162float(A.q[b * A.q_stride + h * D + lane + 32 * e]) * A.scale_log2;
    o[e] = 0.f;
  }
  for (int k = lo + warp; k < end; k += kWarps) {
    const int i = k < P ? k : k - P, max_pages = k < P ? A.max_prompt_pages : A.max_pages, place = i / A.kv.ps;
    const int32_t* table = k < P ? A.prompt_table + (int64_t)g * max_pages : A.table + (int64_t)b * max_pages;
    const int page = page_at(A.kv, table, max_pages, place, A.status);
    if (page < 0) continue;
    const int64_t row = cache_row(A.kv, page, kvh, i - place * A.kv.ps);
    float x = 0.f;
#pragma unroll
    for (int e = 0; e < E; ++e) x = fmaf(q[e], value_at(A.kv.k, A.kv.ks, row, D, lane + 32 * e), x);
#pragma unroll
    for (int s = 16; s > 0; s >>= 1) x += __shfl_xor_sync(0xffffffffu, x, s);
    const float top = fmaxf(m, x), shift = exp2f(m - top), p = exp2f(x - top);
    m = top;
    l = l * shift + p;
#pragma unroll
    for (int e = 0; e < E; ++e) o[e] = o[e] * shift + p * value_at(A.kv.v, A.kv.vs, row, D, lane + 32 * e);
  }
  __shared__ float sm[kWarps], sl[kWarps], so[kWarps][D];
  if (lane == 0) {
    sm[warp] = m;
    sl[warp] = l;
  }
#pragma unroll
  for (int e = 0; e < E; ++e) so[warp][lane + 32 * e] = o[e];
  __syncthreads();
  float top = -INFINITY, total = 0.f;
  for (int w = 0; w < kWarps; ++w) top = fmaxf(top, sm[w]);
  if (top == -INFINITY) top = 0.f;
  for (int w = 0; w < kWarps; ++w) total += sl[w] * exp2f(sm[w] - top);
  for (int d = threadIdx.x; d < D; d += kWarps * 32) {
    float y = 0.f;
    for (int w = 0; w < kWarps; ++w) y += so[w][d] * exp2f(sm[w] - top);
    A.out[((int64_t)b * A.Hq + h) * D + d] = __float2bfloat16(total > 0.f ? y / total : 0.f);
  }
  if (threadIdx.x == 0 && A.lse)
    A.lse[(int64_t)h * A.B + b] = total > 0.f ? (top + log2f(total)) * 0.69314718055994530942f : -INFINITY;
}

template <int CAP>
cudaError_t launch_c(int D, const DecodeArgs& a, const int32_t* groups, cudaStream_t st) {
  const SegTable<CAP> seg = make_segs<CAP>(0, a.G, groups);
  const dim3 grid((unsigned)a.B, (unsigned)a.Hq);
  switch (D) {
    case 64:
      decode_kernel<64, CAP><<<grid, kWarps * 32, 0, st>>>(a, seg);
      break;
    case 128:
      decode_kernel<128, CAP><<<grid, kWarps * 32, 0, st>>>(a, seg);
      break;
    default:
      decode_kernel<512, CAP><<<grid, kWarps * 32, 0, st>>>(a, seg);
  }
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_decode(int D, const DecodeArgs& a, const int32_t* groups, cudaStream_t st) {
  return a.G <= kSmallSegs ? launch_c<kSmallSegs>(D, a, groups, st) : launch_c<kMaxSegs>(D, a, groups, st);
}

size_t decode_workspace_bytes(int, int, int, int) { return 256; }

}  // namespace dkv
