// decode.cuh -- what the kernels of dualkv_decode share: the deal of tiles to workers and the workspace.
#pragma once
#include <stdint.h>

#include "cache.cuh"
#include "kernels.h"
#include "ptx.cuh"
#include "segs.cuh"

namespace dkv {

namespace {

constexpr int kBlocks = 152;    // one per SM
constexpr int kMostShared = 226 << 10;  // dynamic shared memory of a block, 1 KB left for the rest
constexpr float kLowest = -3e38f;  // maximum of a row that has seen nothing: finite, so differences are too

// ---------------------------------------------------------------- the deal
// Tiles of every source in order: prompts 0 .. G - 1, then responses 0 .. B - 1; a source with more rows
// than are taken at once counts its tiles once for every block of rows.  The same sequence follows for each kv-head.
struct Deal {
  uint64_t total, chunk;  // tiles of all kv-heads, and those of one worker: worker w has w chunk .. (w + 1) chunk - 1
  uint32_t per_head;
};
// a / b.  Operands below 2^21 go through fp32, whose quotient is off by 2 units in the last place, so by half at most,
// and its whole part by one (an integer division takes some 250 cycles, and a warp needs five before its first tile).
__device__ __forceinline__ uint32_t divide_small(uint32_t a, uint32_t b) {
  uint32_t q = (uint32_t)__fdividef((float)a, (float)b);
  const int r = (int)a - (int)(q * b);
  if (r < 0) --q;
  if (r >= (int)b) ++q;
  return q;
}
__device__ __forceinline__ uint64_t divide(uint64_t a, uint64_t b) {
  if ((a | b) >> 21 == 0) return divide_small((uint32_t)a, (uint32_t)b);
  return (a | b) >> 32 ? a / b : (uint32_t)a / (uint32_t)b;
}
__device__ __forceinline__ Deal make_deal(uint32_t per_head, int Hkv, int workers) {
  Deal d;
  d.per_head = per_head;
  d.total = (uint64_t)per_head * (uint64_t)Hkv;
  d.chunk = divide(d.total + (uint64_t)workers - 1, (uint64_t)workers);
  return d;
}
__device__ __forceinline__ uint64_t first_tile(const Deal& d, uint32_t worker) {
  const uint64_t at = d.chunk * worker;
  return at < d.total ? at : d.total;
}
__device__ __forceinline__ uint32_t worker_of(const Deal& d, uint64_t tile) { return (uint32_t)divide(tile, d.chunk); }

__device__ __forceinline__ int clamp_len(int n, int max_pages, int ps, uint32_t* status) {
  if (n <= (int64_t)max_pages * ps) return n;
  if (status) atomicOr(status, kDevErrBounds);
  return max_pages * ps;
}
// Prompt of group g (0 without prompts) and tokens of response b (negative: ended), as far as the tables go.
__device__ __forceinline__ int prompt_len(const DecodeArgs& A, int g, uint32_t* status) {
  return A.prompt_lens ? max(0, clamp_len(A.prompt_lens[g], A.max_prompt_pages, A.kv.ps, status)) : 0;
}
__device__ __forceinline__ int response_len(const DecodeArgs& A, int b, uint32_t* status) {
  return clamp_len(A.lens[b], A.max_pages, A.kv.ps, status);
}
// First of the prompt's P tokens that a response of n tokens sees; P if it sees none of them.
__device__ __forceinline__ int first_position(const DecodeArgs& A, int P, int n) {
  return A.window > 0 ? (int)min((int64_t)P, max((int64_t)0, (int64_t)P + n - A.window)) : 0;
}
// Tiles of tokens [lo, end).
template <int TILE>
__device__ __forceinline__ int tiles_of(int lo, int end) {
  return lo < end ? (end + TILE - 1) / TILE - lo / TILE : 0;
}

// A partial result of one row: its maximum (base 2) and sum, and at a source's first tile who goes on with
// the source: `parts` partial results, of this worker (kBlockWorker: a block of prompt.cu) and of those behind it.
constexpr uint32_t kBlockWorker = 0x80000000u;
struct alignas(16) Partial {
  float m, l;
  uint32_t worker;
  int parts;
};
struct Workspace {
  Partial* partial;  // [slots]
  float* o;          // [slots][D] weighted values
};
__host__ __device__ inline size_t align256(size_t x) { return (x + 255) & ~size_t(255); }
// Slots: the rows' own ones of the responses and of the prompts, for a source's first tiles; then those for what a
// worker goes on with that another one began: its rows for each warp of the walk (COLS, by Cfg's warps to a block), and where some
// group may have kBigRows rows, 128 for each block of prompt.cu.
__host__ __device__ constexpr int warp_rows(int D, int GQ) { return D == 512 ? 8 * 8 : GQ > 8 ? 12 * 16 : 16 * 8; }  // of a block
__host__ __device__ inline size_t own_slots(int B, int Hq) { return 2 * (size_t)B * Hq; }
__host__ __device__ inline size_t warp_slots(int D, int GQ) { return (size_t)kBlocks * warp_rows(D, GQ); }
__host__ __device__ inline size_t block_slots(int D, int B, int GQ) {
  return D != 512 && (int64_t)B * GQ >= kBigRows ? (size_t)kBlocks * 128 : 0;
}
__host__ __device__ inline size_t slots_of(int D, int B, int Hq, int GQ) {
  return own_slots(B, Hq) + warp_slots(D, GQ) + block_slots(D, B, GQ);
}
__host__ __device__ inline Workspace carve(void* p, int D, int B, int Hq, int GQ) {
  uint8_t* at = static_cast<uint8_t*>(p);
  Workspace w;
  w.partial = reinterpret_cast<Partial*>(at);
  w.o = reinterpret_cast<float*>(at + align256(sizeof(Partial) * slots_of(D, B, Hq, GQ)));
  return w;
}

// What a block knows of the sources, in shared memory.
struct Sources {
  uint32_t* cum;  // [n + 1] tiles before each source, of one kv-head
  int* len;       // [n] tokens of the prompts (0 .. G - 1) and of the responses (negative: ended)
  int* first;     // [G] first token of the prompt that a response of the group sees; the prompt's length if none does
};

// First token of its own that a response of n tokens sees.
__device__ __forceinline__ int first_own(const DecodeArgs& A, int n) { return A.window > 0 ? max(0, n - A.window) : 0; }

// Tiles that a block of COLS rows of a prompt sees under a window: from the first token that one of its responses does on.
template <int COLS, int TILE, int CAP>
__device__ __forceinline__ int block_tiles(const DecodeArgs& A, const SegTable<CAP>& seg, const Sources& src, int g,
                                           int block) {
  const int GQ = (int)A.by_heads.d, P = src.len[g], row = seg.off[g] * GQ + block * COLS;
  const int last = min(row + COLS, seg.off[g + 1] * GQ) - 1;
  int first = P;
  for (int b = A.by_heads(row); b <= A.by_heads(last); ++b) {
    const int len = src.len[A.G + b];
    if (len >= 0) first = min(first, first_position(A, P, len));
  }
  return tiles_of<TILE>(first, P);
}

// Fills in the above, by the whole block.  BIG: the tiles that prompt.cu's kernel takes, of prompts of groups with kBigRows
// rows and more, n = G; else those of the other prompts and of all responses, n = G + B.  Lengths are kept of all
// sources either way.  Both kernels come to the same decision, from the same numbers.  BLOCKS: under a window, each
// block of a prompt's rows counts its own tiles.
//
// Loops that run a few times, once a launch, are not unrolled here: their instructions come from L2, and a kernel's start waits
// for them (0.3 to 1 us a call).
//
// Few sources: every warp for itself, with two sources to a lane, all of them writing the same, so that no barrier lies
// between a warp and its first tile (32 responses behind one prompt, two such kernels: 52.8 -> 52.0 us).
constexpr int kFewSources = 64, kFewGroups = 8;
template <int COLS, int TILE, bool BIG, bool BLOCKS, int CAP>
__device__ __forceinline__ void deal_few(const DecodeArgs& A, const SegTable<CAP>& seg, const Sources& src) {
  const int G = A.G, all = A.G + A.B, GQ = (int)A.by_heads.d, lane = threadIdx.x & 31;
  int len[2];
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const int i = lane + 32 * k;
    len[k] = i < G ? prompt_len(A, i, A.status) : i < all ? response_len(A, i - G, A.status) : -1;
  }
#pragma unroll
  for (int k = 0; k < 2; ++k)
    if (lane + 32 * k < all) src.len[lane + 32 * k] = len[k];
  __syncwarp();
  unsigned long long work = 0;
#pragma unroll 1
  for (int g = 0; g < G; ++g) {
    uint32_t least = 0x7fffffffu;
#pragma unroll 1
    for (int b = seg.off[g] + lane; b < seg.off[g + 1]; b += 32)
      if (src.len[G + b] >= 0) least = min(least, (uint32_t)src.len[G + b]);
    least = __reduce_min_sync(0xffffffffu, least);
    const int P = src.len[g], rows = (seg.off[g + 1] - seg.off[g]) * GQ;
    const int first = least == 0x7fffffffu ? P : min(P, first_position(A, P, (int)least));
    if (lane == 0) src.first[g] = first;
    if (A.big && rows >= kBigRows) work += (unsigned long long)(P - first) * (unsigned long long)rows;
  }
  __syncwarp();
  const bool big = A.big && work * (unsigned long long)A.kv.Hkv >= big_work(A.kv);
  uint32_t tiles[2];
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const int i = lane + 32 * k;
    tiles[k] = 0;
    if (i < G) {
      const int rows = (seg.off[i + 1] - seg.off[i]) * GQ;
      if (!BLOCKS && (big && rows >= kBigRows) == BIG)
        tiles[k] = (uint32_t)tiles_of<TILE>(src.first[i], len[k]) * (uint32_t)((rows + COLS - 1) / COLS);
    } else if (!BIG && i < all) {
      tiles[k] = (uint32_t)tiles_of<TILE>(first_own(A, len[k]), len[k]) * (uint32_t)((GQ + COLS - 1) / COLS);
    }
  }
  if (BLOCKS) {
#pragma unroll 1
    for (int g = 0; g < G; ++g) {
      const int rows = (seg.off[g + 1] - seg.off[g]) * GQ, blocks = (rows + COLS - 1) / COLS;
      uint32_t n = 0;
      if (!(big && rows >= kBigRows) && src.first[g] < src.len[g])
        for (int i = lane; i < blocks; i += 32) n += (uint32_t)block_tiles<COLS, TILE>(A, seg, src, g, i);
      n = __reduce_add_sync(0xffffffffu, n);
      if (lane == g) tiles[0] = n;
    }
  }
  uint32_t before = 0;
  if (lane == 0) src.cum[0] = 0;
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    uint32_t incl = tiles[k];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t v = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += v;
    }
    if (lane + 32 * k < (BIG ? G : all)) src.cum[1 + lane + 32 * k] = before + incl;
    before += __shfl_sync(0xffffffffu, incl, 31);
  }
  __syncwarp();
}

template <int COLS, int TILE, bool BIG, bool BLOCKS, int CAP>
__device__ __forceinline__ void deal_sources(const DecodeArgs& A, const SegTable<CAP>& seg, const Sources& src,
                                             uint32_t* scratch) {
  __shared__ unsigned long long work;  // tokens times rows of large groups
  if (A.G + A.B <= kFewSources && A.G <= kFewGroups) return deal_few<COLS, TILE, BIG, BLOCKS>(A, seg, src);
  const int G = A.G, n = BIG ? A.G : A.G + A.B, GQ = (int)A.by_heads.d, tid = threadIdx.x, THREADS = blockDim.x;
  const int lane = tid & 31, warp = tid >> 5;
  uint32_t* cum = src.cum;
  if (tid == 0) {
    work = 0;
    cum[0] = 0;
  }
#pragma unroll 2
  for (int i = tid; i < G + A.B; i += THREADS)
    src.len[i] = i < G ? prompt_len(A, i, A.status) : response_len(A, i - G, A.status);
  __syncthreads();
  if (!BIG) {
    const int blocks = (GQ + COLS - 1) / COLS;
    for (int b = tid; b < A.B; b += THREADS) {
      const int len = src.len[G + b];
      cum[1 + G + b] = (uint32_t)tiles_of<TILE>(first_own(A, len), len) * (uint32_t)blocks;
    }
  }
  for (int g = warp; g < G; g += THREADS >> 5) {
    const int from = seg.off[g], to = seg.off[g + 1];
    uint32_t least = 0x7fffffffu;
    for (int b = from + lane; b < to; b += 32) {
      const int len = src.len[G + b];
      if (len >= 0) least = min(least, (uint32_t)len);
    }
    least = __reduce_min_sync(0xffffffffu, least);
    if (lane == 0) {
      const int P = src.len[g], rows = (to - from) * GQ;
      const int first = least == 0x7fffffffu ? P : min(P, first_position(A, P, (int)least));
      src.first[g] = first;
      if (A.big && rows >= kBigRows && first < P)
        atomicAdd(&work, (unsigned long long)(P - first) * (unsigned long long)rows);
    }
  }
  __syncthreads();
  const bool big = A.big && work * (unsigned long long)A.kv.Hkv >= big_work(A.kv);
  if (BLOCKS) {
    for (int g = warp; g < G; g += THREADS >> 5) {
      const int rows = (seg.off[g + 1] - seg.off[g]) * GQ, blocks = (rows + COLS - 1) / COLS;
      uint32_t tiles = 0;
      if (!(big && rows >= kBigRows) && src.first[g] < src.len[g])
        for (int i = lane; i < blocks; i += 32) tiles += (uint32_t)block_tiles<COLS, TILE>(A, seg, src, g, i);
      tiles = __reduce_add_sync(0xffffffffu, tiles);
      if (lane == 0) cum[1 + g] = tiles;
    }
  }
  for (int g = tid; g < G && !BLOCKS; g += THREADS) {
    const int rows = (seg.off[g + 1] - seg.off[g]) * GQ;
    const bool mine = (big && rows >= kBigRows) == BIG;
    cum[1 + g] = mine ? (uint32_t)tiles_of<TILE>(src.first[g], src.len[g]) * (uint32_t)((rows + COLS - 1) / COLS) : 0u;
  }
  __syncthreads();
  // inclusive scan of cum[1 .. n]: every thread takes a run
  const int per = n <= THREADS ? 1 : (n + THREADS - 1) / THREADS, from = 1 + tid * per, to = min(n + 1, from + per);
  uint32_t sum = 0;
  for (int i = from; i < to; ++i) sum += cum[i];
  uint32_t incl = sum;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t v = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += v;
  }
  uint32_t before = incl - sum;
  if (n > 32) {  // else the first warp has them all
    if (lane == 31) scratch[warp] = incl;
    __syncthreads();
    before += __reduce_add_sync(0xffffffffu, lane < warp ? scratch[lane] : 0u);
  }
  for (int i = from; i < to; ++i) {
    before += cum[i];
    cum[i] = before;
  }
  __syncthreads();
}

// Source holding tile `t` of a kv-head: the largest s with cum[s] <= t.
__device__ __forceinline__ int source_of(const uint32_t* cum, int n, uint32_t t) {
  int lo = 0, hi = n - 1;
#pragma unroll 1
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (cum[mid] <= t) lo = mid;
    else hi = mid - 1;
  }
  return lo;
}

}  // namespace

}  // namespace dkv
