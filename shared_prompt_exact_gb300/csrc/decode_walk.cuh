// decode_walk.cuh -- the warps' part of dualkv_decode, compiled without a window (decode.cu) and with one
// (decode_window.cu).
//
// For response b of group g (prompt of P tokens, own n = lens[b] >= 0 tokens, query at P + n - 1):
//   x_k = scale q k over the tokens of the prompt and the response within the window
//   m = max x, l = sum exp(x - m), out = sum exp(x - m) v / l, lse = m + log l
//
// Few queries meet many keys, so the keys' and values' bytes are the bound, each response's read once and each
// prompt's once for its group.  A *source* is a response's own tokens or a group's prompt; its *rows* are the
// queries that see it (the Hq / Hkv heads of a kv-head, of one response or of all of a group).  Sources are cut into tiles
// of 16 to 64 keys, and the tiles of all sources and kv-heads are dealt out in order to the warps of one block per SM, the
// same number to each, whatever the lengths are: a warp walks its share alone, with a running maximum and
// sum per row, and leaves a partial result (sum, maximum, weighted values) for every source that it meets.  The join
// (decode.cu) puts a row's partial results together, its response's and its prompt's, in a fixed order.
// The lengths stay on the device: every block forms the same prefix sum of the sources' tiles.
//
// Inside a warp (mma.m16n8k16, keys as M, up to 8 NT query rows as N):
//   S^T[keys, rows] = K Q^T        K straight from its rows in shared memory as the A operand: the order of the
//                                  head's values in a contraction is free, so a lane takes 16 consecutive bytes
//   O^T[values, rows] += V^T P^T   two keys' words interleaved as the A operand; P^T is the transpose of the
//                                  packed weights (movmatrix); the order of the values is undone when O is written
// Both accumulators have a row's numbers in the same lanes, so a change of its maximum is a product per lane.  Weights are
// rounded to bf16 for their product (2^-9 of each, as in fwd.cu); their sum is taken before.  A tile comes by
// cp.async, keys and values by turns through the warp's own ring: no barrier but the warp's.
//
// Measured: 151 MB of one response in 4 bits in 34 us, 22 us of them the floor.  In its steady state a tile of 64
// keys takes a warp 6,950 cycles, 16 warps to an SM: 0.93 of HBM's rate, with the ALU pipe (4 shifts and
// masks for 8 codes) at two thirds of its own.  A warp's first tile comes after 9,000 cycles: the deal (5,000: two rounds
// of loads and three barriers), the source, its table, its keys.  bf16: 165 MB in 36 us, at HBM's rate behind the start.
#pragma once
#include <cuda_bf16.h>

#include "cache.cuh"
#include "decode.cuh"
#include "kernels.h"
#include "launch.cuh"
#include "ptx.cuh"
#include "segs.cuh"

namespace dkv {

namespace {

constexpr float kRescale = 8.f;    // a maximum moves when a weight would pass 2^8

template <int D, int BITS, int NT>
struct Cfg {
  static constexpr int RB = BITS == 16 ? 2 * D : D / 2;  // bytes of a row
  static constexpr int KP = BITS == 16 ? RB + 16 : RB;   // pitches in shared memory: 16 bytes more where lanes of
  static constexpr int VP = RB + 16;                     // several keys would meet in one bank
  static constexpr int SP = BITS == 16 ? 0 : D / kGroup * 2;  // bytes of a key's scales
  // keys of a tile: 16 for each sub-tile, which lies in one page.  64 in 4 bits cost 5 to 8 % less than 32 (what is done
  // once a tile), bf16 is within 2 % for any tile and ring that leaves 80 KB on their way
  static constexpr int KT = D == 512 ? (BITS == 16 ? 1 : 2) : (BITS == 16 ? (D == 128 ? 2 : 4) : 4);
  static constexpr int TILE = 16 * KT;
  static constexpr int SLOT = TILE * (VP + SP);  // keys or values of a tile, and their scales
  static constexpr int WARPS = D == 512 ? (BITS == 16 ? 6 : 8) : (NT == 2 ? 12 : (BITS == 16 ? 12 : 16));
  static constexpr int SLOTS = D == 64 && BITS == 4 ? 4 : 2;
  static constexpr int COLS = 8 * NT;
  static constexpr int RING = SLOTS * SLOT;  // bytes of a warp's ring
  static_assert(WARPS * COLS <= warp_rows(D, NT == 2 ? 9 : 8), "the workspace has a place for each row of each warp");
};

// Rows that a warp takes at once: 16 where a kv-head has more than 8 and the accumulators leave the registers.
inline int walk_cols(int D, const DecodeArgs& a) { return D != 512 && a.Hq / a.kv.Hkv > 8 ? 16 : 8; }

__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, "
      "%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}
__device__ __forceinline__ void copy16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
template <int WORDS>
__device__ __forceinline__ void load_words(uint32_t (&w)[WORDS], const uint8_t* p) {
  if constexpr (WORDS == 1) {
    w[0] = *reinterpret_cast<const uint32_t*>(p);
  } else if constexpr (WORDS == 2) {
    const uint2 v = *reinterpret_cast<const uint2*>(p);
    w[0] = v.x;
    w[1] = v.y;
  } else {
#pragma unroll
    for (int i = 0; i < WORDS; i += 4) {
      const uint4 v = *reinterpret_cast<const uint4*>(p + 4 * i);
      w[i] = v.x;
      w[i + 1] = v.y;
      w[i + 2] = v.z;
      w[i + 3] = v.w;
    }
  }
}

// ---------------------------------------------------------------- a warp's walk
template <int D, int BITS, int NT, bool WINDOW, int CAP>
__global__ void __launch_bounds__(Cfg<D, BITS, NT>::WARPS * 32, 1)
    decode_kernel(const DecodeArgs A, const __grid_constant__ SegTable<CAP> seg) {
  using C = Cfg<D, BITS, NT>;
  constexpr int TILE = C::TILE, KT = C::KT;
  constexpr int LG = 32 / KT, CPR = C::RB / 16;  // lanes that copy a sub-tile; 16-byte chunks of a row
  const int warps = blockDim.x >> 5;
  extern __shared__ __align__(16) uint8_t smem[];
  const Sources src{reinterpret_cast<uint32_t*>(smem + warps * C::RING),
                    reinterpret_cast<int*>(smem + warps * C::RING) + A.G + A.B + 1,
                    reinterpret_cast<int*>(smem + warps * C::RING) + 2 * (A.G + A.B) + 1};
  const uint32_t* cum = src.cum;
  __shared__ uint32_t scratch[32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, t = lane & 3;
  const int GQ = (int)A.by_heads.d, sources = A.G + A.B;
  const Workspace ws = carve(A.workspace, D, A.B, A.Hq, GQ);
  if (!A.big) cudaGridDependencySynchronize();  // else prompt.cu's kernel has seen to it before this one could start
  deal_sources<C::COLS, C::TILE, false, WINDOW>(A, seg, src, scratch);
  const Deal deal = make_deal(cum[sources], A.kv.Hkv, kBlocks * warps);
  // neighbouring shares go to different SMs, so that a short batch spreads over all of them
  const uint32_t worker = (uint32_t)(warp * kBlocks + blockIdx.x);
  uint64_t at = first_tile(deal, worker);
  const uint64_t stop = first_tile(deal, worker + 1);
  const uint32_t ring = smem_u32(smem) + warp * C::RING;
  uint8_t* ring_p = smem + warp * C::RING;
  // what this lane copies: every LG-th chunk of sub-tile `mine`
  const int mine = lane / LG, li = lane % LG;
  const int copy_row = 16 * mine + (CPR <= LG ? li / CPR : 0), copy_col = CPR <= LG ? li % CPR : li;
  const int step_places = A.by_ps(TILE), step_slots = TILE - step_places * A.kv.ps;

  while (at < stop) {
    // ---- the source, its rows and the tiles of it that are this warp's
    const int kvh = (int)divide(at, deal.per_head);
    const uint32_t local = (uint32_t)(at - (uint64_t)kvh * deal.per_head);
    const int s = source_of(cum, sources, local);
    const bool prompt = s < A.G;
    const int b0 = prompt ? seg.off[s] : s - A.G;
    const int row_begin = b0 * GQ, row_end = (prompt ? seg.off[s + 1] : b0 + 1) * GQ;
    const int blocks = (row_end - row_begin + C::COLS - 1) / C::COLS;
    int tiles = 0, block = 0, t0 = 0;
    if (WINDOW && prompt) {  // the block of rows that has this tile: 32 of them at once
      uint32_t rest = local - cum[s];
      for (int base = 0; base < blocks; base += 32) {
        const uint32_t n = base + lane < blocks ? (uint32_t)block_tiles<C::COLS, TILE>(A, seg, src, s, base + lane) : 0;
        uint32_t incl = n;
#pragma unroll
        for (int i = 1; i < 32; i <<= 1) {
          const uint32_t v = __shfl_up_sync(0xffffffffu, incl, i);
          if (lane >= i) incl += v;
        }
        const uint32_t found = __ballot_sync(0xffffffffu, rest < incl);
        if (found) {
          const int from = __ffs(found) - 1;
          block = base + from;
          tiles = (int)__shfl_sync(0xffffffffu, n, from);
          t0 = (int)(rest - (__shfl_sync(0xffffffffu, incl, from) - (uint32_t)tiles));
          break;
        }
        rest -= __shfl_sync(0xffffffffu, incl, 31);
      }
    } else {
      tiles = (int)divide(cum[s + 1] - cum[s], (uint32_t)blocks);
      block = (int)divide(local - cum[s], (uint32_t)tiles);
      t0 = (int)(local - cum[s]) - block * tiles;
    }
    const int t1 = (int)min((uint64_t)tiles, (uint64_t)t0 + (stop - at));
    const int parts = t0 ? 0 : (int)(worker_of(deal, at + (uint64_t)(tiles - 1)) - worker) + 1;
    at += (uint64_t)(t1 - t0);
    const int r0 = row_begin + block * C::COLS;
    const int end = src.len[s];
    // first tile of the source: its last one ends at `end`
    const int tile0 = (end + TILE - 1) / TILE - tiles;

    // ---- under a window: the first token that each of the lane's rows sees, and the first and last of those of the
    // block's rows
    int lo[WINDOW ? 2 * NT : 1], lo_min = 0, lo_max = 0;
    if (WINDOW) {
      lo_min = 0x7fffffff;
#pragma unroll
      for (int c = 0; c < 2 * NT; ++c) {
        const int r = r0 + 8 * (c >> 1) + 2 * t + (c & 1);
        lo[c] = 0x7fffffff;
        if (r < row_end) {
          const int len = prompt ? src.len[A.G + A.by_heads(r)] : end;
          if (len >= 0) {
            lo[c] = prompt ? first_position(A, end, len) : first_own(A, len);
            lo_min = min(lo_min, lo[c]);
            lo_max = max(lo_max, lo[c]);
          }
        }
      }
      lo_min = __reduce_min_sync(0xffffffffu, lo_min);
      lo_max = __reduce_max_sync(0xffffffffu, lo_max);
    }

    // ---- the producer: keys and values of tiles [first, last) by turns, SLOTS - 1 ahead
    const int first = tile0 + t0, last = tile0 + t1;
    const int max_pages = prompt ? A.max_prompt_pages : A.max_pages;
    const int32_t* table = (prompt ? A.prompt_table : A.table) + (int64_t)(prompt ? s : b0) * max_pages;
    // this lane's sub-tile: its place in the table, its first slot in the page, and the page (loaded a tile ahead)
    int token = first * TILE + 16 * mine, place = A.by_ps(token), in_page = token - place * A.kv.ps;
    int page = first < last && token < end ? table[place] : -1;
    // ---- queries as B operands, in the order in which a lane meets the keys' values (the loads first: they
    // are on their way while the first keys are asked for)
    uint32_t q[NT][D / 16][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const int r = r0 + 8 * nt + g, b = A.by_heads(r);
      const uint4* row = reinterpret_cast<const uint4*>(A.q + b * A.q_stride + (kvh * GQ + (r - b * GQ)) * D);
#pragma unroll
      for (int j = 0; j < D / 32; ++j) {
        const int chunk = BITS == 16 ? 2 * t + (j & 1) + 8 * (j >> 1)
                                     : (D == 64 ? 2 * t + j : 4 * t + 16 * (j >> 2) + (j & 3));
        uint4 w = make_uint4(0, 0, 0, 0);
        if (r < row_end) w = row[chunk];
        q[nt][2 * j][0] = w.x;
        q[nt][2 * j][1] = w.y;
        q[nt][2 * j + 1][0] = w.z;
        q[nt][2 * j + 1][1] = w.w;
      }
    }
    int64_t row = 0;       // of the pools, where the last issued keys' sub-tile starts
    bool has_page = false;
    uint32_t missing = 0;  // tiles in the ring that have a token without a page
    int tile_k = first, tile_v = first, issue_slot = 0;
    auto copy_rows = [&](const void* pool, const __nv_bfloat16* scales, int pitch) {
      const uint32_t dst = ring + issue_slot * C::SLOT;
      const uint8_t* src = static_cast<const uint8_t*>(pool) + row * C::RB + li * 16;
      const uint32_t to = dst + copy_row * pitch + copy_col * 16;
#pragma unroll
      for (int j = 0; j < C::RB / LG; ++j) {
        const int row_j = CPR <= LG ? j * (LG / CPR) : j / (CPR / LG), col_j = CPR <= LG ? 0 : j % (CPR / LG) * LG * 16;
        copy16(to + row_j * pitch + col_j, src + j * LG * 16);
      }
      if (BITS == 4) {
        const uint8_t* sc = reinterpret_cast<const uint8_t*>(scales) + row * C::SP + li * 16;
#pragma unroll
        for (int j = 0; j < (C::SP + LG - 1) / LG; ++j)
          if (li + j * LG < C::SP) copy16(dst + TILE * C::VP + 16 * mine * C::SP + (li + j * LG) * 16, sc + j * LG * 16);
      }
    };
    auto issue_keys = [&]() {
      if (tile_k < last) {
        // sub-tiles in front of every row's window are not looked at: their pages may have been given away
        const bool seen = token < end && (!WINDOW || token + 16 > lo_min);
        has_page = seen && (uint32_t)page < (uint32_t)A.kv.pages;
        const uint32_t bit = 1u << (tile_k & 31);
        missing = __any_sync(0xffffffffu, seen && !has_page) ? missing | bit : missing & ~bit;
        row = cache_row(A.kv, page, kvh, in_page);
        if (has_page) copy_rows(A.kv.k, A.kv.ks, C::KP);
        token += TILE;
        place += step_places;
        in_page += step_slots;
        if (in_page >= A.kv.ps) {
          in_page -= A.kv.ps;
          ++place;
        }
        ++tile_k;
        page = tile_k < last && token < end ? table[place] : -1;
      }
      commit();
      issue_slot = issue_slot == C::SLOTS - 1 ? 0 : issue_slot + 1;
    };
    auto issue_values = [&]() {  // of the tile whose keys were issued last
      if (tile_v < last) {
        if (has_page) copy_rows(A.kv.v, A.kv.vs, C::VP);
        ++tile_v;
      }
      commit();
      issue_slot = issue_slot == C::SLOTS - 1 ? 0 : issue_slot + 1;
    };
    issue_keys();
#pragma unroll
    for (int k = 1; k < C::SLOTS / 2; ++k) {
      issue_values();
      issue_keys();
    }

    if (BITS == 4) {  // values e and e + 4 of each 8 together
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int j = 0; j < D / 32; ++j) {
          uint32_t(&x)[2] = q[nt][2 * j], (&y)[2] = q[nt][2 * j + 1];
          const uint32_t w[4] = {__byte_perm(x[0], y[0], 0x5410), __byte_perm(x[0], y[0], 0x7632),
                                 __byte_perm(x[1], y[1], 0x5410), __byte_perm(x[1], y[1], 0x7632)};
          x[0] = w[0];
          x[1] = w[1];
          y[0] = w[2];
          y[1] = w[3];
        }
    }

    float o[NT][D / 64][4][4], m[NT][2], l[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      m[nt][0] = m[nt][1] = kLowest;
      l[nt][0] = l[nt][1] = 0.f;
#pragma unroll
      for (int i = 0; i < D / 64; ++i)
#pragma unroll
        for (int p = 0; p < 4; ++p)
#pragma unroll
          for (int e = 0; e < 4; ++e) o[nt][i][p][e] = 0.f;
    }

    int slot = 0;
    for (int tile = first; tile < last; ++tile) {
      const int key0 = tile * TILE;
      bool edge = (WINDOW && key0 < lo_max) || key0 + TILE > end;
      // ---- S^T = K Q^T
      wait<C::SLOTS - 2>();
      __syncwarp();
      issue_values();
      uint32_t gone = 0;  // sub-tiles without a page: their keys do not count
      if (missing >> (tile & 31) & 1) {
        const int at_key = key0 + 16 * lane;
        const bool bad = lane < KT && at_key < end && (!WINDOW || at_key + 16 > lo_min) &&
                         page_at(A.kv, table, max_pages, A.by_ps(at_key), A.status) < 0;
        gone = __ballot_sync(0xffffffffu, bad);
        edge = true;
      }
      float sc[KT][NT][4];
      {
        const uint8_t* k = ring_p + slot * C::SLOT;
#pragma unroll
        for (int u = 0; u < KT; ++u) {
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 4; ++e) sc[u][nt][e] = 0.f;
          if constexpr (BITS == 16) {
            const uint8_t* r = k + (16 * u + g) * C::KP + t * 32;
#pragma unroll
            for (int j = 0; j < D / 32; ++j) {
              const int off = 16 * (j & 1) + 128 * (j >> 1);
              const uint4 x = *reinterpret_cast<const uint4*>(r + off);
              const uint4 y = *reinterpret_cast<const uint4*>(r + 8 * C::KP + off);
              const uint32_t a0[4] = {x.x, y.x, x.y, y.y}, a1[4] = {x.z, y.z, x.w, y.w};
#pragma unroll
              for (int nt = 0; nt < NT; ++nt) {
                mma16816(sc[u][nt], a0, q[nt][2 * j][0], q[nt][2 * j][1]);
                mma16816(sc[u][nt], a1, q[nt][2 * j + 1][0], q[nt][2 * j + 1][1]);
              }
            }
          } else {
            constexpr int W = D == 64 ? 2 : 4;  // words that a lane takes at once: within a group of 32
            const uint8_t* r = k + (16 * u + g) * C::KP + 4 * W * t;
            const __nv_bfloat16* scales =
                reinterpret_cast<const __nv_bfloat16*>(k + TILE * C::VP + (16 * u + g) * C::SP) + (D == 64 ? t >> 1 : t);
            const __nv_bfloat162 m24 = __float2bfloat162_rn(-24.f);
#pragma unroll
            for (int j = 0; j < D / (32 * W); ++j) {
              uint32_t x[W], y[W];
              load_words<W>(x, r + 64 * j);
              load_words<W>(y, r + 8 * C::KP + 64 * j);
              const __nv_bfloat162 sx = __bfloat162bfloat162(scales[4 * j]);
              const __nv_bfloat162 sy = __bfloat162bfloat162(scales[4 * j + 8 * (D / kGroup)]);
              const __nv_bfloat162 ox = __hmul2(sx, m24), oy = __hmul2(sy, m24);
#pragma unroll
              for (int w = 0; w < W; ++w) {
                const uint32_t a0[4] = {decode_pair<0>(x[w], sx, ox), decode_pair<0>(y[w], sy, oy),
                                        decode_pair<1>(x[w], sx, ox), decode_pair<1>(y[w], sy, oy)};
                const uint32_t a1[4] = {decode_pair<2>(x[w], sx, ox), decode_pair<2>(y[w], sy, oy),
                                        decode_pair<3>(x[w], sx, ox), decode_pair<3>(y[w], sy, oy)};
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                  mma16816(sc[u][nt], a0, q[nt][2 * (W * j + w)][0], q[nt][2 * (W * j + w)][1]);
                  mma16816(sc[u][nt], a1, q[nt][2 * (W * j + w) + 1][0], q[nt][2 * (W * j + w) + 1][1]);
                }
              }
            }
          }
        }
      }
      slot = slot == C::SLOTS - 1 ? 0 : slot + 1;
      // ---- weights: element e of sc is key g + 8 (e / 2) of its sub-tile, row 2 t + e % 2
      if (edge) {
#pragma unroll
        for (int u = 0; u < KT; ++u)
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const int key = key0 + 16 * u + g + 8 * (e >> 1);
              if ((WINDOW && key < lo[WINDOW ? 2 * nt + (e & 1) : 0]) || key >= end || (gone >> u & 1)) sc[u][nt][e] = -INFINITY;
            }
      }
      float top[NT][2];
      bool grown = false;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          top[nt][c] = fmaxf(sc[0][nt][c], sc[0][nt][c + 2]);
#pragma unroll
          for (int u = 1; u < KT; ++u) top[nt][c] = fmax3(top[nt][c], sc[u][nt][c], sc[u][nt][c + 2]);
          grown |= fmaf(top[nt][c], A.scale_log2, -m[nt][c]) > kRescale;
        }
      if (__any_sync(0xffffffffu, grown)) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            float x = top[nt][c] * A.scale_log2;
#pragma unroll
            for (int i = 4; i < 32; i <<= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, i));
            x = fmaxf(m[nt][c], x);
            const float f = ex2_approx(m[nt][c] - x);
            m[nt][c] = x;
            l[nt][c] *= f;
#pragma unroll
            for (int i = 0; i < D / 64; ++i)
#pragma unroll
              for (int pp = 0; pp < 4; ++pp) {
                o[nt][i][pp][c] *= f;
                o[nt][i][pp][c + 2] *= f;
              }
          }
      }
      uint32_t p[KT][NT][2];
#pragma unroll
      for (int u = 0; u < KT; ++u)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
          for (int e = 0; e < 4; ++e)
            sc[u][nt][e] = ex2_approx(fmaf(sc[u][nt][e], A.scale_log2, -m[nt][e & 1]));
          l[nt][0] += sc[u][nt][0] + sc[u][nt][2];
          l[nt][1] += sc[u][nt][1] + sc[u][nt][3];
          p[u][nt][0] = transpose8x8(pack_bf16x2(sc[u][nt][0], sc[u][nt][1]));
          p[u][nt][1] = transpose8x8(pack_bf16x2(sc[u][nt][2], sc[u][nt][3]));
        }
      // ---- O^T += V^T P^T; this lane's keys are 2 t, 2 t + 1, 2 t + 8, 2 t + 9 of each sub-tile
      wait<C::SLOTS - 2>();
      __syncwarp();
      issue_keys();
      uint8_t* v = ring_p + slot * C::SLOT;
      if (edge) {
        // values that no row sees may be anything: 0 (in 4 bits: their scales), which weights of 0 leave at 0
        for (int k = lane; k < TILE; k += 32) {
          const int key = key0 + k;
          if (key >= lo_min && key < end && !(gone >> (k >> 4) & 1)) continue;
          uint8_t* z = BITS == 16 ? v + k * C::VP : v + TILE * C::VP + k * C::SP;
#pragma unroll 4
          for (int c = 0; c < (BITS == 16 ? C::RB : C::SP) / 4; ++c) reinterpret_cast<uint32_t*>(z)[c] = 0;
        }
        __syncwarp();
      }
#pragma unroll
      for (int u = 0; u < KT; ++u) {
        const uint8_t* r = v + (16 * u + 2 * t) * C::VP;
        if constexpr (BITS == 16) {
          r += 16 * g;
#pragma unroll
          for (int i = 0; i < D / 64; ++i) {
            uint32_t a[4][4];
            load_words<4>(a[0], r + 128 * i);
            load_words<4>(a[1], r + C::VP + 128 * i);
            load_words<4>(a[2], r + 8 * C::VP + 128 * i);
            load_words<4>(a[3], r + 9 * C::VP + 128 * i);
#pragma unroll
            for (int pp = 0; pp < 4; ++pp) {
              const uint32_t f[4] = {__byte_perm(a[0][pp], a[1][pp], 0x5410), __byte_perm(a[0][pp], a[1][pp], 0x7632),
                                     __byte_perm(a[2][pp], a[3][pp], 0x5410), __byte_perm(a[2][pp], a[3][pp], 0x7632)};
#pragma unroll
              for (int nt = 0; nt < NT; ++nt) mma16816(o[nt][i][pp], f, p[u][nt][0], p[u][nt][1]);
            }
          }
        } else {
          constexpr int W = D / 64;  // words of a row in each lane
          const __nv_bfloat16* scales =
              reinterpret_cast<const __nv_bfloat16*>(v + TILE * C::VP + (16 * u + 2 * t) * C::SP) + W * g / 4;
          const __nv_bfloat162 m24 = __float2bfloat162_rn(-24.f);
          uint32_t a[4][W];
#pragma unroll
          for (int k = 0; k < 4; ++k) load_words<W>(a[k], r + ((k & 1) + 8 * (k >> 1)) * C::VP + 4 * W * g);
          __nv_bfloat162 s2[2], o2[2];
#pragma unroll
          for (int w = 0; w < W; ++w) {
            if (w % 4 == 0) {  // a group of 32 values is four words
#pragma unroll
              for (int k = 0; k < 2; ++k) {
                s2[k] = __halves2bfloat162(scales[8 * k * (D / kGroup) + w / 4], scales[(8 * k + 1) * (D / kGroup) + w / 4]);
                o2[k] = __hmul2(s2[k], m24);
              }
            }
            const uint32_t x0 = __byte_perm(a[0][w], a[1][w], 0x5410), x1 = __byte_perm(a[0][w], a[1][w], 0x7632);
            const uint32_t y0 = __byte_perm(a[2][w], a[3][w], 0x5410), y1 = __byte_perm(a[2][w], a[3][w], 0x7632);
#define DKV_PV(E)                                                                                             \
  {                                                                                                           \
    const uint32_t f[4] = {decode_pair<E>(x0, s2[0], o2[0]), decode_pair<E>(x1, s2[0], o2[0]),                \
                           decode_pair<E>(y0, s2[1], o2[1]), decode_pair<E>(y1, s2[1], o2[1])};               \
    _Pragma("unroll") for (int nt = 0; nt < NT; ++nt) mma16816(o[nt][w][E], f, p[u][nt][0], p[u][nt][1]);     \
  }
            DKV_PV(0)
            DKV_PV(1)
            DKV_PV(2)
            DKV_PV(3)
#undef DKV_PV
          }
        }
      }
      slot = slot == C::SLOTS - 1 ? 0 : slot + 1;
    }
    __syncwarp();

    // ---- the partial result: the source's own places if its first tile is here, else this warp's
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        float sum = l[nt][c];
#pragma unroll
        for (int x = 4; x < 32; x <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, x);
        const int col = 8 * nt + 2 * t + c, r = r0 + col;
        if (r >= row_end) continue;
        const int b = A.by_heads(r);
        const size_t rows = (size_t)A.B * A.Hq;
        const size_t to = t0 == 0 ? (prompt ? rows : 0) + (size_t)b * A.Hq + kvh * GQ + (r - b * GQ)
                                  : own_slots(A.B, A.Hq) + (size_t)worker * C::COLS + col;
        if (g == 0) ws.partial[to] = Partial{m[nt][c], sum, worker, parts};
        float* out = ws.o + to * D;
#pragma unroll
        for (int i = 0; i < D / 64; ++i) {
          const auto& x = o[nt][i];
          // bf16: values 2 pp and 2 pp + 1 of the chunk; 4 bits: pp and pp + 4 of the word
          float4* dst = reinterpret_cast<float4*>(out + (BITS == 16 ? 8 * g + 64 * i : 8 * (D / 64 * g + i)));
          if (BITS == 16) {
            dst[0] = make_float4(x[0][c], x[0][c + 2], x[1][c], x[1][c + 2]);
            dst[1] = make_float4(x[2][c], x[2][c + 2], x[3][c], x[3][c + 2]);
          } else {
            dst[0] = make_float4(x[0][c], x[1][c], x[2][c], x[3][c]);
            dst[1] = make_float4(x[0][c + 2], x[1][c + 2], x[2][c + 2], x[3][c + 2]);
          }
        }
      }
  }
  // the kernel of the large groups' prompts may still run: the join, which waits for this one, needs both
  if (warp == 0) cudaGridDependencySynchronize();
}

template <int D, int BITS, int NT, bool WINDOW, int CAP>
cudaError_t walk_c(const DecodeArgs& a, const int32_t* groups, cudaStream_t st) {
  using C = Cfg<D, BITS, NT>;
  const SegTable<CAP> seg = make_segs<CAP>(0, a.G, groups);
  // many sources take the place of some warps' rings
  const int sources = (3 * a.G + 2 * a.B + 1) * (int)sizeof(uint32_t), room = (kMostShared - sources) / C::RING;
  const int warps = room < C::WARPS ? room : C::WARPS, smem = warps * C::RING + sources;
  const cudaError_t e = allow_shared<&decode_kernel<D, BITS, NT, WINDOW, CAP>>(a.device, kMostShared);
  if (e != cudaSuccess) return e;
  return launch_behind_shared(decode_kernel<D, BITS, NT, WINDOW, CAP>, dim3(kBlocks), dim3(warps * 32), smem, st, a, seg);
}
template <int D, int BITS, bool WINDOW>
cudaError_t walk_b(const DecodeArgs& a, const int32_t* groups, cudaStream_t st) {
  const bool few = a.G <= kSmallSegs;
  if constexpr (D != 512) {
    if (walk_cols(D, a) == 16)
      return few ? walk_c<D, BITS, 2, WINDOW, kSmallSegs>(a, groups, st) : walk_c<D, BITS, 2, WINDOW, kMaxSegs>(a, groups, st);
  }
  return few ? walk_c<D, BITS, 1, WINDOW, kSmallSegs>(a, groups, st) : walk_c<D, BITS, 1, WINDOW, kMaxSegs>(a, groups, st);
}
template <bool WINDOW>
cudaError_t walk(int D, const DecodeArgs& a, const int32_t* groups, cudaStream_t st) {
  const bool four = a.kv.ks != nullptr;
  switch (D) {
    case 64:
      return four ? walk_b<64, 4, WINDOW>(a, groups, st) : walk_b<64, 16, WINDOW>(a, groups, st);
    case 128:
      return four ? walk_b<128, 4, WINDOW>(a, groups, st) : walk_b<128, 16, WINDOW>(a, groups, st);
    case 512:
      return four ? walk_b<512, 4, WINDOW>(a, groups, st) : walk_b<512, 16, WINDOW>(a, groups, st);
    default:
      return cudaErrorInvalidValue;
  }
}

}  // namespace

}  // namespace dkv
