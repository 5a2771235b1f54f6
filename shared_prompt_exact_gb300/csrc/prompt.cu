// prompt.cu -- the prompt's part of dualkv_decode for groups with many rows.
//
// A group's rows for one kv-head (its responses' heads: 32 responses of 4 heads are 128) see the same prompt, so
// this is a product of matrices: 128 rows meet tiles of 128 keys on the tensor cores (tcgen05), as
// in fwd.cu's forward of head dimensions 64 and 128.  What differs: keys and values come from pages, a block
// takes an equal share of all prompts' tiles (decode.cuh's deal; whole_chunk), and it leaves partial results,
// fp32 values with a row's maximum and sum, which decode.cu's join puts together with the responses'.
//
// Warps:
//   loaders of keys, loaders of values, each with a ring of their own.  bf16: one warp each, 8 lanes of which load a
//     tile's 16-token pieces by TMA, each from its page.  4 bits: four warps each; a thread decodes
//     a row (its codes loaded a tile ahead) and writes them as bf16 in the swizzled layout that TMA would leave.  The decoded
//     order within 8 values is 0, 4, 1, 5, ... (decode8); the queries are written in the same order, and the
//     output's columns are put right at the end.
//   an issuer of S = Q K^T, an issuer of O += P V, eight softmax warps: as in fwd.cu.
// Measured, alone and from cold caches: 25 MB of one prompt of 6,144 tokens for 128 rows of 8 kv-heads in 18.7 us (14 behind
// other calls), six prompts of 3,000 tokens in 4 bits in 28.8.  A block needs 15,000 cycles to its first scores (5,000 of them the deal; then its pages, its first keys, which
// all blocks ask for at once), 1,000 a tile in bf16 and 2,200 in 4 bits (issue: the loaders' 250 instructions a row and
// the softmax's 350 a tile share the schedulers; two loader warps an operand instead of four: 5,000), and 6,000 at its end,
// where 64 KB of partial results go through 16 KB of shared memory so that rows are written in 64-byte runs (a row to
// a lane: 2,000 more).
// Values that no row sees may hold anything: rows of a tile outside the prompt or before its first seen token are
// written as zeros by the loaders themselves.
#include <cuda.h>
#include <cuda_bf16.h>

#include "cache.cuh"
#include "decode.cuh"
#include "kernels.h"
#include "launch.cuh"
#include "ptx.cuh"
#include "segs.cuh"

namespace dkv {

namespace {

template <int D, int BITS>
struct PromptCfg {
  static constexpr int BM = 128, BN = 128, HC = 64;
  static constexpr int QCH = D / 64;                    // 64-column chunks of a row
  static constexpr int TILE_BYTES = QCH * BN * 128;
  static constexpr int NK = 3, NV = 2;                  // tiles in the rings of keys and of values
  static constexpr int LW = BITS == 16 ? 1 : 4;         // loader warps of each
  static constexpr int V_WARP = LW, SOFTMAX = BITS == 16 ? 4 : 8;  // the first of eight softmax warps
  static constexpr int S_WARP = BITS == 16 ? 2 : 16, PV_WARP = S_WARP + 1;
  static constexpr int THREADS = BITS == 16 ? 384 : 640;
  static constexpr int OFF_K = TILE_BYTES, OFF_V = OFF_K + NK * TILE_BYTES, RINGS = OFF_V + NV * TILE_BYTES;
  static constexpr int MOST_SHARED = RINGS + 1024 + (4 * kBigGroups + kBigResponses + 2) * (int)sizeof(uint32_t);
  static constexpr uint32_t TM_S = 0, TM_O = 256, TM_COLS = 512;
  static constexpr float RESCALE_THRESHOLD = 8.0f;  // log2 units
};

struct PromptCtl {
  uint64_t k_full[3], k_empty[3], v_full[2], v_empty[2];
  uint64_t q_full, q_free, s_full[2], p_full[2], pv_done[2], pv_issued[2], pair_done[4], drain, drain2;
  uint32_t tmem_base;
  int abort_flag;
  uint32_t chunk;
  uint32_t scratch[32];
  float half_m[256], half_l[256];
};

__device__ __forceinline__ void fence_async() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

template <int N>
__device__ __forceinline__ void registers_up() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void registers_down() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}

// A warp's wait; its lanes go on, or give up, together.
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, const FailState& fs) {
  return __all_sync(0xffffffffu, mbar_wait(bar, parity, fs));
}

// Tiles of a chunk so that no block has parts of two pieces (a piece: a prompt, kv-head and block of rows), each piece
// filled up to a multiple of the chunk with tiles that nobody forms.  A block that goes on to another piece waits for its
// partial results and its new queries, as long as for MORE tiles; 0 if no chunk up to so much larger than the mean, d.chunk,
// leaves enough blocks for it.  One warp; lane i tries d.chunk + i.
// Whole calls, 32/8 heads of 128: one prompt of 5,000 tokens for 32 responses 33 -> 27 us, two of 8,000 in 4 bits for
// 64/8 heads 88 -> 74.  The search costs 1 us where nothing is to be filled up (6,144 tokens: 52.3 -> 52.9).  MORE = 6 is slower
// (twelve prompts of 1,000 to 3,000: 96 us, not 93), and without a bound eight prompts of 300 to 9,000 take 179, not 120.
template <int MORE, int CAP>
__device__ __forceinline__ uint32_t whole_chunk(const DecodeArgs& A, const SegTable<CAP>& seg, const Sources& src,
                                                const Deal& d, uint32_t* padded) {
  const int G = A.G, Hkv = A.kv.Hkv, lane = threadIdx.x & 31;
  if (G > kBlocks || d.chunk == 0 || (d.chunk | src.cum[G]) >> 20) return 0;
  const uint32_t c = (uint32_t)d.chunk + lane;
  uint32_t n = 0;
#pragma unroll 1
  for (int g = 0; g < G; ++g) {
    if (src.cum[g + 1] == src.cum[g]) continue;
    const uint32_t blocks = (uint32_t)((seg.off[g + 1] - seg.off[g]) * (int)A.by_heads.d + 127) / 128;
    n += blocks * divide_small((uint32_t)tiles_of<128>(src.first[g], src.len[g]) + c - 1, c);
  }
  const uint32_t fits = __ballot_sync(0xffffffffu, lane <= MORE && n * (uint64_t)Hkv <= kBlocks);
  if (!fits) return 0;
  const uint32_t chunk = (uint32_t)d.chunk + __ffs(fits) - 1;
  uint32_t before = 0;
#pragma unroll 1
  for (int g = 0; g < G; ++g) {
    if (lane == 0) padded[g] = before;
    if (src.cum[g + 1] == src.cum[g]) continue;
    const uint32_t blocks = (uint32_t)((seg.off[g + 1] - seg.off[g]) * (int)A.by_heads.d + 127) / 128;
    before += blocks * chunk * divide_small((uint32_t)tiles_of<128>(src.first[g], src.len[g]) + chunk - 1, chunk);
  }
  if (lane == 0) padded[G] = before;
  return chunk;
}

// One prompt, kv-head and block of 128 rows: the tiles of it that are this block's.
struct Segment {
  int g, kvh, r0, row_end, P, lo, first, last;
  int parts;   // blocks that have a part of it, this one and those behind, if its first tile is here; else 0
};

template <int D, int BITS, int CAP>
__global__ void __launch_bounds__(PromptCfg<D, BITS>::THREADS, 1)
    prompt_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV, const DecodeArgs A,
                  const __grid_constant__ SegTable<CAP> seg) {
  using C = PromptCfg<D, BITS>;
  constexpr int QCH = C::QCH;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  __shared__ PromptCtl ctl;
  const Sources src{reinterpret_cast<uint32_t*>(smem + C::RINGS), reinterpret_cast<int*>(smem + C::RINGS) + 2 * A.G + 1,
                    reinterpret_cast<int*>(smem + C::RINGS) + A.G + 1};
  const uint32_t warp = __shfl_sync(0xffffffffu, warp_id(), 0), lane = lane_id();
  const int GQ = (int)A.by_heads.d, ps = A.kv.ps;
  FailState fs{&ctl.abort_flag, A.status, A.wait_limit_ns};

  if (threadIdx.x == 0) {
    ctl.abort_flag = 0;
    for (int i = 0; i < C::NK; ++i) {
      mbar_init(&ctl.k_full[i], C::LW);
      mbar_init(&ctl.k_empty[i], 1);
    }
    for (int i = 0; i < C::NV; ++i) {
      mbar_init(&ctl.v_full[i], C::LW);
      mbar_init(&ctl.v_empty[i], 1);
    }
    mbar_init(&ctl.q_full, 256);
    mbar_init(&ctl.q_free, 8);
    for (int i = 0; i < 2; ++i) {
      mbar_init(&ctl.s_full[i], 1);
      mbar_init(&ctl.p_full[i], 8);
      mbar_init(&ctl.pv_done[i], 1);
      mbar_init(&ctl.pv_issued[i], 1);
    }
    for (int i = 0; i < 4; ++i) mbar_init(&ctl.pair_done[i], 64);
    mbar_init(&ctl.drain, 1);
    mbar_init(&ctl.drain2, 1);
    fence_mbar_init();
  }
  if (warp == C::S_WARP) {
    tmem_alloc(&ctl.tmem_base, C::TM_COLS);
    tmem_relinquish();
  }
  tc_fence_before();
  cudaGridDependencySynchronize();
  deal_sources<128, 128, true, false>(A, seg, src, ctl.scratch);
  uint32_t* padded = src.cum + 3 * A.G + A.B + 1;  // [G + 1] tiles before each prompt, with those that fill up its pieces
  Deal deal = make_deal(src.cum[A.G], A.kv.Hkv, kBlocks);
  if (warp == 0) {
    const uint32_t chunk = whole_chunk<3>(A, seg, src, deal, padded);
    if (lane == 0) ctl.chunk = chunk;
  }
  __syncthreads();
  tc_fence_after();
  cudaTriggerProgrammaticLaunchCompletion();  // the responses' kernel may start where SMs are free
  const uint32_t tmem = ctl.tmem_base;
  const Workspace ws = carve(A.workspace, D, A.B, A.Hq, GQ);
  const uint32_t* cum = src.cum;
  if (ctl.chunk) {
    cum = padded;
    deal.per_head = cum[A.G];
    deal.total = (uint64_t)deal.per_head * (uint64_t)A.kv.Hkv;
    deal.chunk = ctl.chunk;
  }
  const uint64_t begin = first_tile(deal, blockIdx.x), stop = first_tile(deal, blockIdx.x + 1);
  auto next_segment = [&](uint64_t& at) {
    Segment s;
    s.kvh = (int)divide(at, deal.per_head);
    const uint32_t local = (uint32_t)(at - (uint64_t)s.kvh * deal.per_head);
    s.g = source_of(cum, A.G, local);
    const int begin_row = seg.off[s.g] * GQ;
    s.row_end = seg.off[s.g + 1] * GQ;
    const int blocks = (s.row_end - begin_row + C::BM - 1) / C::BM;
    s.P = src.len[s.g];
    s.lo = src.first[s.g];
    const int tile0 = s.lo / C::BN, tiles = tiles_of<C::BN>(s.lo, s.P);
    const uint32_t all = cum[s.g + 1] - cum[s.g], from = local - cum[s.g];
    const int room = blocks == 1 ? (int)all : (int)divide(all, (uint32_t)blocks);
    const int block = blocks == 1 ? 0 : (int)divide(from, (uint32_t)room), t0 = (int)from - block * room;
    const int t1 = (int)min((uint64_t)tiles, (uint64_t)t0 + (stop - at));
    s.parts = t0 ? 0 : (int)(worker_of(deal, at + (uint64_t)(tiles - 1)) - blockIdx.x) + 1;
    at += (uint64_t)((t1 == tiles ? room : t1) - t0);
    s.r0 = begin_row + block * C::BM;
    s.first = tile0 + t0;
    s.last = tile0 + t1;
    return s;
  };
  // the table's entry for a token, -1 behind the prompt: to be held against the pool's pages where it is used, a tile
  // later, so that nothing waits for its load
  auto entry_of = [&](const Segment& s, int token) {
    return token < s.P ? A.prompt_table[(int64_t)s.g * A.max_prompt_pages + A.by_ps(token)] : -1;
  };
  auto is_page = [&](int entry) { return (uint32_t)entry < (uint32_t)A.kv.pages; };

  // 4 bits: 20 warps start with 96 registers a thread; the softmax warps take over what the others leave:
  // 2 x 72 + 2 x 144 + 48 for the five warpgroups, 5 x 96 in all
  if (warp < 2 * C::LW) {
    // ------------------------------------------------------------ loaders
    if (BITS == 4) registers_down<72>();
    const bool values = warp >= C::V_WARP;
    const int slots = values ? C::NV : C::NK;
    uint64_t* full = values ? ctl.v_full : ctl.k_full;
    uint64_t* empty = values ? ctl.v_empty : ctl.k_empty;
    uint8_t* ring = smem + (values ? C::OFF_V : C::OFF_K);
    int slot = 0;
    uint32_t phase = 1;  // parity of the wait for the slot's previous reader: passes at once in the first round
    int filled = 0;
    bool ok = true;
    if constexpr (BITS == 16) {
      const CUtensorMap* tm = values ? &tmV : &tmK;
      if (lane == 0) tma_prefetch_desc(tm);
      for (uint64_t at = begin; at < stop && ok;) {
        const Segment s = next_segment(at);
        int token = s.first * C::BN + 16 * (int)(lane & 7), page = entry_of(s, token);
        for (int tile = s.first; tile < s.last; ++tile) {
          const bool have = lane < 8 && is_page(page);
          const bool whole = have && (!values || (token >= s.lo && token + 16 <= s.P));
          const int row = have ? (int)cache_row(A.kv, page, s.kvh, token - A.by_ps(token) * ps) : 0;
          token += C::BN;
          const int next = tile + 1 < s.last ? entry_of(s, token) : -1;
          if (!(ok = warp_wait(&empty[slot], phase, fs))) break;
          uint8_t* dst = ring + slot * C::TILE_BYTES;
          const uint32_t boxes = __ballot_sync(0xffffffffu, whole), have_mask = __ballot_sync(0xffffffffu, have);
          if (values && boxes != 0xffu) {  // pieces with tokens that no row sees: zeros in their place
            for (int piece = 0; piece < 8; ++piece) {
              if (boxes >> piece & 1) continue;
              const int64_t row0 = __shfl_sync(0xffffffffu, row, piece);
              const int key0 = tile * C::BN + 16 * piece;
              for (int i = (int)lane; i < 16 * 8 * QCH; i += 32) {
                const int r = i / (8 * QCH), c = i % (8 * QCH), key = key0 + r;
                uint4 x = make_uint4(0, 0, 0, 0);
                if ((have_mask >> piece & 1) && key >= s.lo && key < s.P)
                  x = reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(A.kv.v) + (row0 + r) * (2 * D))[c];
                *reinterpret_cast<uint4*>(dst + (c >> 3) * C::BN * 128 + sw128_offset(16 * piece + r, c & 7)) = x;
              }
            }
            fence_async();
            __syncwarp();
          }
          const bool skip = !values && filled == A.test_skip_tile;  // failure-path self-test: never loaded
          if (lane == 0 && !skip) mbar_arrive_expect_tx(&full[slot], __popc(boxes) * 16 * 128 * QCH);
          __syncwarp();
          if (whole && !skip)
            for (int c = 0; c < QCH; ++c)
              tma_load_3d(dst + c * C::BN * 128 + lane * 16 * 128, tm, &full[slot], c * 64, 0, row);
          page = next;
          ++filled;
          if (++slot == slots) {
            slot = 0;
            phase ^= 1;
          }
        }
      }
      // copies still in flight end before the block does
      if (!ok)
        for (int back = 1; back <= slots && back <= filled; ++back) {
          if (!values && filled - back == A.test_skip_tile) continue;
          mbar_wait_drain(&full[(filled - back) % slots], ((filled - back) / slots) & 1, kWaitLimitNs);
        }
    } else {
      constexpr int U = D / 32;  // 16-byte vectors of a row's codes: one for each group of 32 values
      const int mine = (int)(warp - (values ? C::V_WARP : 0)) * 32 + (int)lane;  // this thread's row of a tile
      const uint8_t* pool = static_cast<const uint8_t*>(values ? A.kv.v : A.kv.k);
      const __nv_bfloat16* scales = values ? A.kv.vs : A.kv.ks;
      struct Row {
        uint4 codes[U];
        __nv_bfloat162 sc[U / 2];
      };
      int page = -1;  // table's entry for this row in the tile that `load` takes next
      auto find = [&](const Segment& s, int tile) {
        const int token = tile * C::BN + mine;
        page = tile < s.last && token >= s.lo ? entry_of(s, token) : -1;
      };
      auto load = [&](Row& x, const Segment& s, int tile) {  // then finds the page for the next one
        const int token = tile * C::BN + mine;
#pragma unroll
        for (int u = 0; u < U; ++u) x.codes[u] = make_uint4(0, 0, 0, 0);
#pragma unroll
        for (int u = 0; u < U / 2; ++u) x.sc[u] = __float2bfloat162_rn(0.f);
        if (is_page(page)) {
          const int64_t row = cache_row(A.kv, page, s.kvh, token - A.by_ps(token) * ps);
          const uint4* from = reinterpret_cast<const uint4*>(pool + row * (D / 2));
          const __nv_bfloat162* sf = reinterpret_cast<const __nv_bfloat162*>(scales + row * U);
#pragma unroll
          for (int u = 0; u < U; ++u) x.codes[u] = from[u];
#pragma unroll
          for (int u = 0; u < U / 2; ++u) x.sc[u] = sf[u];
        }
        find(s, tile + 1);
      };
      auto decode = [&](const Row& x) {
        if (!(ok = warp_wait(&empty[slot], phase, fs))) return;
        uint8_t* dst = ring + slot * C::TILE_BYTES;
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const __nv_bfloat162 s2 = u & 1 ? __high2bfloat162(x.sc[u / 2]) : __low2bfloat162(x.sc[u / 2]);
          const __nv_bfloat162 o2 = __hmul2(s2, __float2bfloat162_rn(-24.f));
          const uint32_t w[4] = {x.codes[u].x, x.codes[u].y, x.codes[u].z, x.codes[u].w};
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int c = 4 * u + i;  // 16-byte chunk of the row
            *reinterpret_cast<uint4*>(dst + (c >> 3) * C::BN * 128 + sw128_offset(mine, c & 7)) = decode8(w[i], s2, o2);
          }
        }
        fence_async();
        __syncwarp();
        if (lane == 0 && (values || filled != A.test_skip_tile)) mbar_arrive(&full[slot]);
        ++filled;
        if (++slot == slots) {
          slot = 0;
          phase ^= 1;
        }
      };
      Row x, y;  // codes of two tiles, on their way while the ones before are decoded
      for (uint64_t at = begin; at < stop && ok;) {
        const Segment s = next_segment(at);
        find(s, s.first);
        load(x, s, s.first);
        for (int tile = s.first; tile < s.last && ok; tile += 2) {
          load(y, s, tile + 1);
          decode(x);
          if (tile + 1 >= s.last || !ok) break;
          load(x, s, tile + 2);
          decode(y);
        }
      }
    }
  } else if (warp >= C::SOFTMAX && warp < C::SOFTMAX + 8) {
    // ------------------------------------------------------------ softmax
    if (BITS == 4) registers_up<144>();
    const uint32_t wq = warp & 3;
    const int half = (int)(warp - C::SOFTMAX) >> 2, row = (int)(wq * 32 + lane);
    const uint32_t tl = tmem + ((wq * 32) << 16), tO = tl + C::TM_O + half * D;
    const float sl2 = A.scale_log2;
    bool ok = true;
    int jj = 0, n_seg = 0;
    for (uint64_t at = begin; at < stop && ok; ++n_seg) {
      const Segment s = next_segment(at);
      // ---- this thread's half of its query; every product with the previous ones has been waited for
      const int r = s.r0 + row, b_of = A.by_heads(r), head = s.kvh * GQ + (r - b_of * GQ);
      int lo = 0x7fffffff;  // first token that the row sees
      // the queries go where other warps may still pass on their partial results
      if (n_seg > 0 && !(ok = warp_wait(&ctl.q_free, (n_seg - 1) & 1, fs))) break;
      {
        // the warp's 16 rows, D / 8 lanes to a row
        constexpr int LR = D / 8, AT_ONCE = 32 / LR;
        const int first_row = (int)(warp - C::SOFTMAX) * 16 + (int)lane / LR, c = (int)lane % LR;
        uint4 x[16 / AT_ONCE];
#pragma unroll
        for (int i = 0; i < 16 / AT_ONCE; ++i) {
          const int rr = s.r0 + first_row + i * AT_ONCE, bb = A.by_heads(rr);
          x[i] = make_uint4(0, 0, 0, 0);
          if (rr < s.row_end)
            x[i] = reinterpret_cast<const uint4*>(A.q + bb * A.q_stride + (int64_t)(s.kvh * GQ + rr - bb * GQ) * D)[c];
        }
#pragma unroll
        for (int i = 0; i < 16 / AT_ONCE; ++i) {
          uint4 y = x[i];
          if (BITS == 4)  // values e and e + 4 together, as decode8 leaves them
            y = make_uint4(__byte_perm(y.x, y.z, 0x5410), __byte_perm(y.x, y.z, 0x7632), __byte_perm(y.y, y.w, 0x5410),
                           __byte_perm(y.y, y.w, 0x7632));
          *reinterpret_cast<uint4*>(smem + (c >> 3) * C::BM * 128 + sw128_offset(first_row + i * AT_ONCE, c & 7)) = y;
        }
        if (r < s.row_end) {
          const int len = src.len[A.G + b_of];
          if (len >= 0) lo = first_position(A, s.P, len);
        }
        fence_async();
        mbar_arrive(&ctl.q_full);
      }
      float m = -INFINITY, l = 0.f;
      for (int tile = s.first; tile < s.last; ++tile, ++jj) {
        const uint32_t b = jj & 1;
        const int kl0 = tile * C::BN + half * C::HC;
        const int clo = lo - kl0, chi = s.P - 1 - kl0;  // allowed columns [clo, chi] of this half
        // 16-token pieces of the half without a page: their keys do not count
        const int piece = kl0 + 16 * (int)(lane & 3);
        const uint32_t gone = __ballot_sync(0xffffffffu, lane < 4 && piece < s.P && piece + 15 >= s.lo && !is_page(entry_of(s, piece)));
        if (gone && lane == 0 && A.status) atomicOr(A.status, kDevErrBounds);
        const bool full = clo <= 0 && chi >= C::HC - 1 && !gone;
        if (!(ok = warp_wait(&ctl.s_full[b], (jj >> 1) & 1, fs))) break;
        tc_fence_after();
        float x[C::HC];
#pragma unroll
        for (int c4 = 0; c4 < C::HC / 32; ++c4) {
          uint32_t rr[32];
          tmem_ld32(tl + C::TM_S + b * C::BN + half * C::HC + c4 * 32, rr);
#pragma unroll
          for (int i = 0; i < 32; ++i) x[c4 * 32 + i] = __uint_as_float(rr[i]);
        }
        tmem_ld_wait();
        if (!full) {
#pragma unroll
          for (int c = 0; c < C::HC; ++c) x[c] = (c < clo || c > chi || (gone >> (c >> 4) & 1)) ? -INFINITY : x[c];
        }
        float mq[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
        for (int c = 0; c < C::HC; c += 8) {
#pragma unroll
          for (int q4 = 0; q4 < 4; ++q4) mq[q4] = fmax3(mq[q4], x[c + 2 * q4], x[c + 2 * q4 + 1]);
        }
        const float mx = fmax3(fmaxf(mq[0], mq[1]), mq[2], mq[3]);
        const float m_new = fmaxf(m, mx * sl2);  // -inf stays -inf (sl2 > 0)
        if (tile == s.first) {
          m = m_new;
        } else if (__any_sync(0xffffffffu, m_new > m + C::RESCALE_THRESHOLD)) {
          const float alpha = (m_new == -INFINITY) ? 1.f : ex2_approx(m - m_new);
          if (!(ok = warp_wait(&ctl.pv_done[(jj - 1) & 1], ((jj - 1) >> 1) & 1, fs))) break;
          tc_fence_after();
#pragma unroll
          for (int c4 = 0; c4 < D / 32; ++c4) {
            uint32_t rr[32];
            tmem_ld32(tO + c4 * 32, rr);
            tmem_ld_wait();
#pragma unroll
            for (int i = 0; i < 32; ++i) rr[i] = __float_as_uint(__uint_as_float(rr[i]) * alpha);
            tmem_st32(tO + c4 * 32, rr);
          }
          tmem_st_wait();
          l *= alpha;
          m = m_new;
        }
        const float m_use = (m == -INFINITY) ? 0.f : m;
        const float2 sl2v = make_float2(sl2, sl2), negm = make_float2(-m_use, -m_use);
        float2 sum2[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
        uint32_t w[32];
#pragma unroll
        for (int e = 0; e < 32; ++e) {
          const float2 y = ffma2(make_float2(x[2 * e], x[2 * e + 1]), sl2v, negm);
          const float2 pp = make_float2(ex2_approx(y.x), ex2_approx(y.y));
          sum2[e & 1] = fadd2(sum2[e & 1], pp);
          w[e] = pack_bf16x2(pp.x, pp.y);
        }
        tmem_st32(tl + C::TM_S + b * C::BN + half * C::HC, w);
        const float2 st = fadd2(sum2[0], sum2[1]);
        l += st.x + st.y;
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&ctl.p_full[b]);
      }
      if (!ok) break;
      // ---- the halves' sums relative to one maximum -> the row's partial result
      if (!(ok = warp_wait(&ctl.pv_done[(jj - 1) & 1], ((jj - 1) >> 1) & 1, fs))) break;
      tc_fence_after();
      ctl.half_m[half * 128 + row] = m;
      ctl.half_l[half * 128 + row] = l;
      mbar_arrive(&ctl.pair_done[wq]);
      if (!(ok = warp_wait(&ctl.pair_done[wq], n_seg & 1, fs))) break;
      const float m0 = ctl.half_m[row], m1 = ctl.half_m[128 + row], l0 = ctl.half_l[row], l1 = ctl.half_l[128 + row];
      const float mtot = fmaxf(m0, m1), mref = mtot == -INFINITY ? kLowest : mtot;
      const float f0 = m0 == -INFINITY ? 0.f : ex2_approx(m0 - mref), f1 = m1 == -INFINITY ? 0.f : ex2_approx(m1 - mref);
      const size_t own = own_slots(A.B, A.Hq);
      const size_t to = s.parts ? own / 2 + (size_t)b_of * A.Hq + head : own + warp_slots(D, GQ) + (size_t)blockIdx.x * 128 + row;
      constexpr int OC = D / 2;  // output columns of this thread
      // 16 columns at a time through 2 KB of the queries' place (their products are done), so that 4 lanes write
      // 64 bytes of one row; the rows' slots are consecutive but where a response's other heads lie between
      float* stage = reinterpret_cast<float*>(smem) + (warp - C::SOFTMAX) * 512;
      const uint32_t slot_lo = (uint32_t)to, slot_hi = (uint32_t)(to >> 32), live = __ballot_sync(0xffffffffu, r < s.row_end);
#pragma unroll
      for (int c4 = 0; c4 < OC / 32; ++c4) {
        uint32_t u0[32], u1[32];
        tmem_ld32(tl + C::TM_O + half * OC + c4 * 32, u0);
        tmem_ld32(tl + C::TM_O + D + half * OC + c4 * 32, u1);
        tmem_ld_wait();
        float y[32];
#pragma unroll
        for (int i = 0; i < 32; ++i) {
          const int d = BITS == 4 ? (i & ~7) | ((i & 7) >> 1) | ((i & 1) << 2) : i;  // column i is value d
          y[d] = fmaf(__uint_as_float(u1[i]), f1, __uint_as_float(u0[i]) * f0);
        }
#pragma unroll
        for (int c2 = 0; c2 < 2; ++c2) {
#pragma unroll
          for (int i = 0; i < 4; ++i)  // four 16-byte vectors a row, at places that differ from row to row
            *reinterpret_cast<float4*>(stage + lane * 16 + ((i ^ (lane >> 1)) & 3) * 4) =
                make_float4(y[16 * c2 + 4 * i], y[16 * c2 + 4 * i + 1], y[16 * c2 + 4 * i + 2], y[16 * c2 + 4 * i + 3]);
          __syncwarp();
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const int from = 8 * k + (int)(lane >> 2), i = lane & 3;
            const float4 x = *reinterpret_cast<const float4*>(stage + from * 16 + ((i ^ (from >> 1)) & 3) * 4);
            const size_t at_slot = (size_t)__shfl_sync(0xffffffffu, slot_lo, from) |
                                   (size_t)__shfl_sync(0xffffffffu, slot_hi, from) << 32;
            if (live >> from & 1)
              *reinterpret_cast<float4*>(ws.o + at_slot * D + half * OC + c4 * 32 + c2 * 16 + i * 4) = x;
          }
          __syncwarp();
        }
      }
      if (lane == 0) mbar_arrive(&ctl.q_free);
      if (r < s.row_end && half == 0) ws.partial[to] = Partial{mref, l0 * f0 + l1 * f1, kBlockWorker | blockIdx.x, s.parts};
    }
  } else {
    if (BITS == 4) registers_down<48>();  // the whole warpgroup, idle warps too
    if (warp == C::S_WARP) {
      // ------------------------------------------------------------ S issuer
      constexpr uint32_t idS = idesc_bf16(128, C::BN, 0, 0);
      const uint64_t qdesc = sdesc_sw128(smem_u32(smem), 16, 1024);
      const uint32_t ring = smem_u32(smem + C::OFF_K);
      bool ok = true;
      int jj = 0, n_seg = 0;
      for (uint64_t at = begin; at < stop && ok; ++n_seg) {
        const Segment s = next_segment(at);
        if (!(ok = warp_wait(&ctl.q_full, n_seg & 1, fs))) break;
        for (int tile = s.first; tile < s.last; ++tile, ++jj) {
          const uint32_t b = jj & 1, tS = tmem + C::TM_S + b * C::BN;
          const int slot = jj % C::NK;
          if (jj >= 2 && !(ok = warp_wait(&ctl.pv_issued[b], ((jj >> 1) - 1) & 1, fs))) break;
          if (!(ok = warp_wait(&ctl.k_full[slot], (jj / C::NK) & 1, fs))) break;
          tc_fence_after();
          const uint64_t kdesc = sdesc_sw128(ring + slot * C::TILE_BYTES, 16, 1024);
          if (elect_one()) {
  #pragma unroll
            for (int c = 0; c < QCH; ++c)
  #pragma unroll
              for (int k = 0; k < 4; ++k)
                mma_bf16_ss(tS, sdesc_add(qdesc, c * C::BM * 128 + k * 32), sdesc_add(kdesc, c * C::BN * 128 + k * 32), idS,
                            (c | k) != 0);
            mma_commit(&ctl.k_empty[slot]);
            mma_commit(&ctl.s_full[b]);
          }
          __syncwarp();
        }
      }
      if (begin < stop) {  // every MMA issued above ends before TMEM is released
        if (elect_one()) mma_commit(&ctl.drain);
        __syncwarp();
        mbar_wait_drain(&ctl.drain, 0, kWaitLimitNs);
      }
    } else if (warp == C::PV_WARP) {
      // ------------------------------------------------------------ PV issuer
      constexpr uint32_t idO = idesc_bf16(128, D, 0, 1);
      const uint32_t ring = smem_u32(smem + C::OFF_V);
      bool ok = true;
      int jj = 0;
      for (uint64_t at = begin; at < stop && ok;) {
        const Segment s = next_segment(at);
        for (int tile = s.first; tile < s.last; ++tile, ++jj) {
          const uint32_t b = jj & 1, tP = tmem + C::TM_S + b * C::BN, acc0 = tile > s.first ? 1u : 0u;
          const int slot = jj % C::NV;
          if (!(ok = warp_wait(&ctl.p_full[b], (jj >> 1) & 1, fs))) break;
          if (!(ok = warp_wait(&ctl.v_full[slot], (jj / C::NV) & 1, fs))) break;
          tc_fence_after();
          const uint64_t vdesc = sdesc_sw128(ring + slot * C::TILE_BYTES, C::BN * 128, 1024);
          if (elect_one()) {
  #pragma unroll
            for (int h = 0; h < 2; ++h)
  #pragma unroll
              for (int k = 0; k < C::HC / 16; ++k)
                mma_bf16_ts(tmem + C::TM_O + h * D, tP + h * C::HC + k * 8, sdesc_add(vdesc, (h * C::HC + k * 16) * 128), idO,
                            k > 0 ? 1u : acc0);
            mma_commit(&ctl.v_empty[slot]);
            mma_commit(&ctl.pv_done[b]);
          }
          __syncwarp();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&ctl.pv_issued[b]);
        }
      }
      if (begin < stop) {
        if (elect_one()) mma_commit(&ctl.drain2);
        __syncwarp();
        mbar_wait_drain(&ctl.drain2, 0, kWaitLimitNs);
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == C::S_WARP) tmem_dealloc(tmem, C::TM_COLS);
}

template <int D, int BITS, int CAP>
cudaError_t launch_t(const DecodeArgs& a, const CUtensorMap& tk, const CUtensorMap& tv, const int32_t* groups,
                     cudaStream_t st) {
  using C = PromptCfg<D, BITS>;
  const SegTable<CAP> seg = make_segs<CAP>(0, a.G, groups);
  const int smem = C::RINGS + 1024 + (4 * a.G + a.B + 2) * (int)sizeof(uint32_t);
  const cudaError_t e = allow_shared<&prompt_kernel<D, BITS, CAP>>(a.device, C::MOST_SHARED);
  if (e != cudaSuccess) return e;
  return launch_behind_shared(prompt_kernel<D, BITS, CAP>, dim3(kBlocks), dim3(C::THREADS), smem, st, tk, tv, a, seg);
}

template <int D, int BITS>
cudaError_t launch_b(const DecodeArgs& a, const CUtensorMap& tk, const CUtensorMap& tv, const int32_t* groups,
                     cudaStream_t st) {
  return a.G <= kSmallSegs ? launch_t<D, BITS, kSmallSegs>(a, tk, tv, groups, st)
                           : launch_t<D, BITS, kMaxSegs>(a, tk, tv, groups, st);
}

}  // namespace

cudaError_t launch_prompt(int D, const DecodeArgs& a, const CUtensorMap& tk, const CUtensorMap& tv, const int32_t* groups,
                          cudaStream_t st) {
  const bool four = a.kv.ks != nullptr;
  if (D == 64) return four ? launch_b<64, 4>(a, tk, tv, groups, st) : launch_b<64, 16>(a, tk, tv, groups, st);
  if (D == 128) return four ? launch_b<128, 4>(a, tk, tv, groups, st) : launch_b<128, 16>(a, tk, tv, groups, st);
  return cudaErrorInvalidValue;
}

}  // namespace dkv
