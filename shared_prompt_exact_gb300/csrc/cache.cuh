// cache.cuh -- the paged key/value cache as the kernels see it.
//
// A cache is two pools of pages, keys and values; a page holds ps consecutive tokens of
// every kv-head: row (page, head, slot) has D values, head by head, so ps tokens of one
// head are contiguous.  With 16 bits a value is a bf16; with 4 bits it is scale * (code - 8):
// codes two to a byte (the even value in the low half) and one bf16 scale for every 32 values.
// A stream's tokens lie in the pages that its row of a page table names, ps to a page in order.
#pragma once
#include <cuda_bf16.h>
#include <stdint.h>

#include "kernels.h"
#include "ptx.cuh"

namespace dkv {

constexpr int kGroup = 32;  // values that share a scale

// Page of token `index` (>= 0) in a stream's row of the table, or -1 (recorded in the status word)
// where the table has none or names one outside the pool: nothing is read or written through it.
__device__ __forceinline__ int page_at(const PagedKV& kv, const int32_t* table, int max_pages, int place,
                                       uint32_t* status) {
  int page = -1;
  if (place < max_pages) page = table[place];
  if ((uint32_t)page < (uint32_t)kv.pages) return page;
  if (status) atomicOr(status, kDevErrBounds);
  return -1;
}

// Row of the pools for (page, head, slot).
__device__ __forceinline__ int64_t cache_row(const PagedKV& kv, int page, int head, int slot) {
  return ((int64_t)page * kv.Hkv + head) * kv.ps + slot;
}

// (x & mask) | bits in one instruction (with both constants as immediates it becomes two).
__device__ __forceinline__ uint32_t and_or(uint32_t x, uint32_t mask, uint32_t bits) {
  uint32_t r;
  asm("lop3.b32 %0, %1, %2, %3, 0xea;" : "=r"(r) : "r"(x), "r"(mask), "r"(bits));
  return r;
}

// Codes E and E + 4 of the 8 in w as their values: 16 + code has the code in the mantissa's top four bits, and
// (16 + code) s - 24 s = (code - 8) s is exact in bf16, since scales have 5 significant bits (24 s has 7 at most,
// the result 8).
template <int E>
__device__ __forceinline__ uint32_t decode_pair(uint32_t w, __nv_bfloat162 s, __nv_bfloat162 minus24s) {
  const uint32_t u = and_or(E == 0 ? w << 3 : w >> (E == 0 ? 0 : 4 * E - 3), 0x00780078u, 0x41804180u);
  const __nv_bfloat162 r = __hfma2(*reinterpret_cast<const __nv_bfloat162*>(&u), s, minus24s);
  return *reinterpret_cast<const uint32_t*>(&r);
}
// All 8 codes of w: 0 and 4, 1 and 5, 2 and 6, 3 and 7.
__device__ __forceinline__ uint4 decode8(uint32_t w, __nv_bfloat162 s, __nv_bfloat162 minus24s) {
  return make_uint4(decode_pair<0>(w, s, minus24s), decode_pair<1>(w, s, minus24s), decode_pair<2>(w, s, minus24s),
                    decode_pair<3>(w, s, minus24s));
}

}  // namespace dkv
