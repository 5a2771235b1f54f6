// decode.cu -- dualkv_decode: attention of one new token per response over the paged cache.  The prompts of large groups go
// to prompt.cu's blocks, everything else to the warps of decode_walk.cuh; both leave partial results, which the
// kernel here joins.
#include "decode_walk.cuh"

namespace dkv {

namespace {

// ---------------------------------------------------------------- the join
constexpr int kJoinWarps = 16;  // most warps of a block

// Bound by latency: the row's own two partial results say how many others there are and where; then those, 8 to a warp
// at once.  300 of them a row (32 rows) in 7.6 us, 7 (6,144 rows) in 9; with every warp working its row's places out from the
// deal it was 20 and 14.
// `share` warps take a row's partial results by turns, some at once with their loads together; each keeps a running
// maximum, and the first of them joins what they have.  The kernel may start before the partial results are
// complete, so nothing that reads them is __restrict__.
template <int D, int CAP>
__global__ void __launch_bounds__(kJoinWarps * 32)
    join_kernel(const DecodeArgs A, int share, int cols, const __grid_constant__ SegTable<CAP> seg) {
  constexpr int E = D / 64, BATCH = D == 512 ? 2 : 8;  // float2s of a lane; partial results on their way at once
  __shared__ float2 sums[kJoinWarps][D / 2];
  __shared__ float2 ml[kJoinWarps];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, part = warp & (share - 1);
  const int64_t row = (int64_t)blockIdx.x * ((blockDim.x >> 5) / share) + warp / share;
  const bool live = row < (int64_t)A.B * A.Hq;
  const int b = live ? (int)(row / A.Hq) : 0, h = live ? (int)(row - (int64_t)b * A.Hq) : 0;
  const int GQ = (int)A.by_heads.d, j = h - A.by_heads(h) * GQ, g = seg_of(seg, b);
  const Workspace ws = carve(A.workspace, D, A.B, A.Hq, GQ);
  // which sources the row sees, as the kernels that left the partial results decided (who wrote the lengths was complete
  // before those began, so they may be read before the wait)
  const int len = response_len(A, b, nullptr), P = prompt_len(A, g, nullptr);
  const bool sees_own = live && len > 0, sees_prompt = live && len >= 0 && first_position(A, P, len) < P;
  const size_t own = own_slots(A.B, A.Hq);
  const int in_group = (b - seg.off[g]) * GQ + j;
  cudaGridDependencySynchronize();
  const Partial none{kLowest, 0.f, 0, 0};
  Partial p0 = sees_prompt ? ws.partial[own / 2 + row] : none, p1 = sees_own ? ws.partial[row] : none;
  // A block of prompt.cu's whose wait ran out has left nothing, and what lies in its place may be anything: workers without
  // places in the workspace are recorded and count as none.
  auto hold = [&](Partial& p) {
    const bool block = p.worker & kBlockWorker;
    const size_t end = (size_t)(p.worker & ~kBlockWorker) + (size_t)max(p.parts, 0);
    if (p.parts >= 1 && end * (size_t)(block ? 128 : cols) <= (block ? block_slots(D, A.B, GQ) : warp_slots(D, GQ))) return;
    if (A.status) atomicOr(A.status, kDevErrBounds);
    p = none;
  };
  if (sees_prompt) hold(p0);
  if (sees_own) hold(p1);
  const bool big = p0.worker & kBlockWorker;
  const int n = p0.parts + p1.parts;
  // slots of the workers behind a source's first one
  const size_t behind0 = big ? own + warp_slots(D, GQ) + (size_t)(p0.worker & ~kBlockWorker) * 128 + (in_group & 127)
                             : own + (size_t)p0.worker * cols + (in_group & (cols - 1));
  const size_t behind1 = own + (size_t)p1.worker * cols + (j & (cols - 1));
  auto place = [&](int i) {
    const bool second = i >= p0.parts;
    const int k = second ? i - p0.parts : i;
    if (k == 0) return second ? (size_t)row : own / 2 + (size_t)row;
    return (second ? behind1 : behind0) + (size_t)(k * (second || !big ? cols : 128));
  };
  float top = kLowest, total = 0.f;
  float2 acc[E];
#pragma unroll
  for (int e = 0; e < E; ++e) acc[e] = make_float2(0.f, 0.f);
  for (int i0 = part; i0 < n; i0 += BATCH * share) {
    float2 f[BATCH], v[BATCH][E];
#pragma unroll
    for (int k = 0; k < BATCH; ++k) {
      const int i = i0 + k * share;
      f[k] = make_float2(kLowest, 0.f);
#pragma unroll
      for (int e = 0; e < E; ++e) v[k][e] = make_float2(0.f, 0.f);
      if (i < n) {
        const size_t at = place(i);
        f[k] = *reinterpret_cast<const float2*>(&ws.partial[at]);
#pragma unroll
        for (int e = 0; e < E; ++e) v[k][e] = reinterpret_cast<const float2*>(ws.o + at * D)[lane + 32 * e];
      }
    }
    float most = top;
#pragma unroll
    for (int k = 0; k < BATCH; ++k) most = fmaxf(most, f[k].x);
    const float old = ex2_approx(top - most);
    top = most;
    total *= old;
#pragma unroll
    for (int e = 0; e < E; ++e) acc[e] = fmul2(acc[e], make_float2(old, old));
#pragma unroll
    for (int k = 0; k < BATCH; ++k) {
      const float w = ex2_approx(f[k].x - most);
      total = fmaf(f[k].y, w, total);
#pragma unroll
      for (int e = 0; e < E; ++e) acc[e] = ffma2(v[k][e], make_float2(w, w), acc[e]);
    }
  }
  if (share > 1) {
#pragma unroll
    for (int e = 0; e < E; ++e) sums[warp][lane + 32 * e] = acc[e];
    if (lane == 0) ml[warp] = make_float2(top, total);
    __syncthreads();
    if (part) return;
    float most = top;
    for (int w = 1; w < share; ++w) most = fmaxf(most, ml[warp + w].x);
    const float mine = ex2_approx(top - most);
    top = most;
    total *= mine;
#pragma unroll
    for (int e = 0; e < E; ++e) acc[e] = fmul2(acc[e], make_float2(mine, mine));
#pragma unroll 4
    for (int w = 1; w < share; ++w) {
      const float2 x = ml[warp + w];
      const float f = ex2_approx(x.x - most);
      total = fmaf(x.y, f, total);
#pragma unroll
      for (int e = 0; e < E; ++e) acc[e] = ffma2(sums[warp + w][lane + 32 * e], make_float2(f, f), acc[e]);
    }
  }
  if (!live) return;
  const float inv = total == 0.f ? 0.f : 1.f / total;  // 0: nothing seen; NaN stays NaN, here and in lse
  uint32_t* out = reinterpret_cast<uint32_t*>(A.out + row * D);
#pragma unroll
  for (int e = 0; e < E; ++e) out[lane + 32 * e] = pack_bf16x2(acc[e].x * inv, acc[e].y * inv);
  if (lane == 0 && A.lse)
    A.lse[(int64_t)h * A.B + b] = total == 0.f ? -INFINITY : (top + log2f(total)) * 0.69314718055994530942f;
}

template <int D, int CAP>
cudaError_t join_c(const DecodeArgs& a, const int32_t* groups, cudaStream_t st) {
  const SegTable<CAP> seg = make_segs<CAP>(0, a.G, groups);
  // few rows can have many partial results each: as many warps to a row as there are warps for, in blocks of 4 or more
  const int64_t rows = (int64_t)a.B * a.Hq, spare = kBlocks * kJoinWarps / rows;
  const int share = spare >= 16 ? 16 : spare >= 8 ? 8 : spare >= 4 ? 4 : spare >= 2 ? 2 : 1, per = share < 4 ? 4 / share : 1;
  return launch_behind(join_kernel<D, CAP>, dim3((unsigned)((rows + per - 1) / per)), dim3(per * share * 32), st, a, share,
                       walk_cols(D, a), seg);
}
template <int D>
cudaError_t join(const DecodeArgs& a, const int32_t* groups, cudaStream_t st) {
  return a.G <= kSmallSegs ? join_c<D, kSmallSegs>(a, groups, st) : join_c<D, kMaxSegs>(a, groups, st);
}

}  // namespace

cudaError_t launch_decode(int D, const DecodeArgs& a, const CUtensorMap& tk, const CUtensorMap& tv, const int32_t* groups,
                          cudaStream_t st) {
  cudaError_t e = a.big ? launch_prompt(D, a, tk, tv, groups, st) : cudaSuccess;
  if (e == cudaSuccess) e = a.window > 0 ? launch_walk_window(D, a, groups, st) : walk<false>(D, a, groups, st);
  if (e != cudaSuccess) return e;
  return D == 64 ? join<64>(a, groups, st) : D == 128 ? join<128>(a, groups, st) : join<512>(a, groups, st);
}

size_t decode_workspace_bytes(int B, int Hq, int Hkv, int D) {
  const Workspace w = carve(nullptr, D, B, Hq, Hq / Hkv);
  return reinterpret_cast<size_t>(w.o) + sizeof(float) * slots_of(D, B, Hq, Hq / Hkv) * (size_t)D;
}

}  // namespace dkv
