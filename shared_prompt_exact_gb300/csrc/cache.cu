// cache.cu -- new rows of keys and values into a paged cache, and rows of it back.
//
// append: for row t of stream s, the (t - off[s])-th of the n_s rows of this call, with lens[s]
// tokens held afterwards:
//   index i = lens[s] - n_s + (t - off[s]),  position p = starts[s] + i
//   q, k: per-head norm and rotation by p f_j as in rope.cu;  q -> q_out,  k and v -> (page i / ps, slot i % ps)
//   4 bits, for each 32 values of a head:
//     step = max |x| / 7 rounded up to 5 significant bits (so (code - 8) step is exact in bf16)
//     n = x / step rounded to the nearest, ties away from zero;  code = n + 8
//     a group with a value that is not finite gets the scale NaN
// read: the same rows back in bf16.
//
// Codes and steps jump at borders, so which arithmetic a key comes from shows.  4-bit keys are what fp32 gives, each operation
// rounded once:
//   m = mean x^2 (of its exact value), r = rsqrt(m + eps), a = (x r) (w + w0), c and s = cosine and sine of the angle in 64 bits,
//   key = (a c) - (b s) or (b c) + (a s);  step = ceil5(max |key| / 7), n = floor(|key| / step + 1/2)
// so that any fp32 program in that order finds the same codes, but for the last bit of its mean.  The kernel forms them in the
// order that is fastest (rope.cu's) and knows the error of that (kKeyError): a group with a border that near is formed
// again, in this order (settle_group).
//
// Both touch each value once and are bound by HBM bandwidth (few rows: by latency).  The walk over
// rows and heads, the loads ahead through shared memory and the arithmetic are rope.cu's: one warp per
// row, q's heads first, then k's, then v's.  Keys are quantised before any rounding to bf16.
// Measured: append of 71,680 rows of 32 + 2 x 8 heads of 128 in bf16 267 us (6.6 TB/s); of 23,200 rows of 8 + 2 x 2 heads of
// 512 in 4 bits 98 us (5.1 TB/s: bound by issue, 2,860 instructions a row; 90 us without the look at borders, of which
// 4 are its instructions and 4 the groups formed again, in 2 % of the steps: 2.7 us for a warp's first one; in fp64 it was 7 us and the
// launch 120; with a bound 8 times as small 95 us); read of 131,072 rows of 8 heads of 128 156 us (6.9 TB/s; 177 with the
// values asked for behind the keys).
#include <cuda_bf16.h>

#include "cache.cuh"
#include "kernels.h"
#include "launch.cuh"
#include "ptx.cuh"
#include "rope.cuh"
#include "segs.cuh"
#include "twofloat.cuh"

namespace dkv {

namespace {

constexpr int kWarps = 8;
constexpr int kThreads = kWarps * 32;
constexpr int kDepth = 3;  // steps in a lane's ring, as in rope.cu
constexpr int kResident = 152 * 2;  // blocks of the append that the GPU holds

// Where a row of the call goes: its position, its slot in a page, and the table's entry for that page, which is
// held against the pool where it is used (-1: there is none).
struct Place {
  uint32_t pos;
  int slot, entry;
};
// The stream's numbers for row t, and from them the row's place: two loads behind one another, so a warp that has
// several rows asks for each a row ahead.
struct StreamOf {
  int s, len, start;
};
template <int CAP>
__device__ __forceinline__ StreamOf stream_of(const SegTable<CAP>& seg, const int32_t* lens, const int32_t* starts, int64_t t,
                                              int64_t T) {
  StreamOf x{0, 0, 0};
  if (t >= T) return x;
  x.s = seg_of(seg, (int)t);
  x.len = lens[x.s];
  if (starts) x.start = starts[x.s];
  return x;
}
template <int CAP>
__device__ __forceinline__ Place place_of(const StreamOf& x, const FastDiv& by_ps, const SegTable<CAP>& seg,
                                          const int32_t* table, int max_pages, int64_t t, int64_t T) {
  Place p{0, 0, -1};
  if (t >= T) return p;
  const int index = x.len - (seg.off[x.s + 1] - (int)t);
  p.pos = (uint32_t)x.start + (uint32_t)index;
  if (index < (int)t - seg.off[x.s]) return p;  // the stream is said to hold fewer tokens than this call has of it
  const int page = by_ps(index);
  p.slot = index - page * (int)by_ps.d;
  if (page < max_pages) p.entry = table[(int64_t)x.s * max_pages + page];
  return p;
}
__device__ __forceinline__ bool has_page(const PagedKV& kv, const Place& p, uint32_t* status) {
  if ((uint32_t)p.entry < (uint32_t)kv.pages) return true;
  if (status) atomicOr(status, kDevErrBounds);
  return false;
}

// A group of keys whose codes the walk's arithmetic does not decide: group `group` of head `head` in row t at position pos,
// bound for row `row` of the pool.
struct Undecided {
  int64_t row;
  int t, head, group;
  uint32_t pos;
};

// What a block of the append keeps in shared memory.
template <int D, int BITS>
struct AppendShared {
  alignas(16) float w[2][D];
  alignas(16) float cs[kWarps][D / 2];
  alignas(16) float sn[kWarps][D / 2];
  uint64_t freq[D / 2];
  alignas(16) float k[BITS == 4 ? kWarps : 1][BITS == 4 ? 512 : 4];  // a step's keys, Vec8s in their order
  alignas(8) float size[BITS == 4 ? kWarps : 1][BITS == 4 ? 64 : 2];  // of every 8: largest magnitude around, 0: exact
  uint4 ring[kDepth][2][kThreads];
};

// Largest magnitude of three, NaN if one of them is.
__device__ __forceinline__ float magnitude3(float a, float b, float c) {
  float r;
  asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
__device__ __forceinline__ float magnitude8(const Vec8& x) {
  return magnitude3(magnitude3(magnitude3(x.v[0].x, x.v[0].y, x.v[1].x), x.v[1].y, x.v[2].x),
                    magnitude3(x.v[2].y, x.v[3].x, x.v[3].y), 0.f);
}

// Difference between a key as the walk forms it and as it is defined, by the largest magnitude of the two vectors that its lane
// turned, with u = 2^-24.  The walk: sum of squares 14 u, + eps u, root half of that and 4 u, product with the weight 3 u: 14.5 u of each
// value of a pair; cosine and sine 1.6 u for the angle's float and 4 u; their products' roundings 2 u: in all 16.5 u sqrt(2) +
// 5.6 u * 2 = 35 u.  The definition: mean and eps u, root 4 u, products and weight 3 u, cosine and sine, their products
// and sum 3 u: 11 u sqrt(2) = 16 u.
constexpr float kKeyError = 52.f * 0x1p-24f;

// x rounded up to 5 significant bits.
__device__ __forceinline__ uint32_t five_bits(float x) { return (__float_as_uint(x) + 0x7ffffu) & ~0x7ffffu; }

// Codes of 16 consecutive values; the neighbouring lane holds the other 16 of the group.  `size`: 0 where the values are bf16
// as they came, else the magnitude that their errors go by (kKeyError); then `near` is set where an error could change a
// code or the scale.
template <bool KEYS>
__device__ __forceinline__ uint2 quantise16(Vec8 (&x)[2], float size, __nv_bfloat16& scale, bool& near) {
  const float most = magnitude3(magnitude8(x[0]), magnitude8(x[1]), 0.f);
  const float top = magnitude3(most, __shfl_xor_sync(0xffffffffu, most, 1), most);
  const float t = __fdiv_rn(top, 7.f);
  const uint32_t bits = five_bits(t);
  const bool finite = top < __uint_as_float(0x7f800000u);  // false for NaN
  scale = __ushort_as_bfloat16((unsigned short)(finite ? bits >> 16 : 0x7fc0u));
  near = false;
  if (KEYS) {
    const float around = magnitude3(size, __shfl_xor_sync(0xffffffffu, size, 1), size);
    const float off = fmaf(around, kKeyError / 7.f, t * 0x1p-22f);
    near = finite && around != 0.f && five_bits(fmaxf(t - off, 0.f)) != five_bits(t + off);  // a NaN around: true
  }
  if (!finite || bits == 0u) return make_uint2(0x88888888u, 0x88888888u);  // not finite, or zeros
  // x / step by the reciprocal.  bf16 values take the smallest float above it: one half way comes out above (away
  // from zero) and goes to the farther multiple, any other is moved by 2^-23 of it at most, less than it is away from half
  // way.  Others take the nearest float, which moves them by 2^-24.  The sum with 1.5 x 2^23 + 8 is rounded to
  // a whole number, whose low bits are n + 8; the eight codes are shifted together with the upper bits in place,
  // which are subtracted at once.
  float step = __uint_as_float(bits);
  if (step < 1e-36f) {  // its reciprocal could overflow: the same with everything 2^64 times as large
    step *= 0x1p64f;
    size *= 0x1p64f;
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e / 4].v[e % 4] = fmul2(x[e / 4].v[e % 4], make_float2(0x1p64f, 0x1p64f));
  }
  const bool exact = !KEYS || size == 0.f;
  const float inv = exact ? __uint_as_float(__float_as_uint(__frcp_rd(step)) + 1u) : __frcp_rn(step);
  const float2 inv2 = make_float2(inv, inv), minus = make_float2(-inv, -inv), magic = make_float2(12582920.f, 12582920.f);
  uint32_t out[2];
  float far = 0.f;  // from the nearest multiple, in steps
#pragma unroll
  for (int w = 0; w < 2; ++w) {
    float2 n[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      n[e] = ffma2(x[w].v[e], inv2, magic);
      if (KEYS) {
        const float2 d = ffma2(x[w].v[e], minus, fadd2(n[e], make_float2(-12582920.f, -12582920.f)));
        far = magnitude3(far, d.x, d.y);
      }
    }
    const float codes[8] = {n[0].x, n[2].x, n[0].y, n[2].y, n[1].x, n[3].x, n[1].y, n[3].y};
    uint32_t sum = 0;
#pragma unroll
    for (int e = 7; e >= 0; --e) sum = (sum << 4) + __float_as_uint(codes[e]);
    out[w] = sum - 0x4b400000u * 0x11111111u;
  }
  // (2^-20: the reciprocal's error of 7 2^-24 here, the quotient's and the sum's of 4 2^-24 each in the definition)
  if (KEYS) near |= !exact && !(far <= 0.5f - fmaf(size, kKeyError * inv, 0x1p-20f));
  return make_uint2(out[0], out[1]);
}

// The rotation of the lane's values that are turned; the others pass as they are, infinities among them.
__device__ __forceinline__ void turn(Vec8& a, Vec8& b, const Angles& g, const LaneMap& m, bool inter) {
  if (!inter) {
    if (m.ta) rotate(a, b, g.cs, g.sn, g.neg, false);
    return;
  }
  if (m.ta) {
    turn2(a.v[0], a.v[2], g.cs.v[0], g.sn.v[0], g.neg.v[0]);
    turn2(a.v[1], a.v[3], g.cs.v[1], g.sn.v[1], g.neg.v[1]);
  }
  if (m.tb) {
    turn2(b.v[0], b.v[2], g.cs.v[2], g.sn.v[2], g.neg.v[2]);
    turn2(b.v[1], b.v[3], g.cs.v[3], g.sn.v[3], g.neg.v[3]);
  }
}

// Place of value p (a multiple of 4) of a step's 512 in shared memory: vectors of 16 bytes, so that neither the lanes that
// write neighbouring ones nor those that read every fourth meet in a bank.
__device__ __forceinline__ int spread(int p) { return p ^ ((p >> 5 & 3) << 2); }
__device__ __forceinline__ void store8(const Vec8& v, float* base, int p) {
  *reinterpret_cast<float4*>(base + spread(p)) = make_float4(v.v[0].x, v.v[0].y, v.v[1].x, v.v[1].y);
  *reinterpret_cast<float4*>(base + spread(p + 4)) = make_float4(v.v[2].x, v.v[2].y, v.v[3].x, v.v[3].y);
}

// A lane's 16 codes into a row of the 4-bit pools.
template <int D>
__device__ __forceinline__ void store_codes(const uint2& c, __nv_bfloat16 scale, void* codes, __nv_bfloat16* scales, int64_t row,
                                            int i) {
  *reinterpret_cast<uint2*>(static_cast<uint8_t*>(codes) + row * (D / 2) + 8 * i) = c;
  if ((i & 1) == 0) scales[row * (D / kGroup) + i / 2] = scale;
}

// One group of 32 keys from its row of k, a value to a lane, as the keys' definition has them (above): codes and scale into the
// pool.  The sum of squares and the cosines and sines come from two floats, rounded once.
template <int D>
__device__ __noinline__ void settle_group(const AppendArgs& A, const uint64_t* freq, const Undecided& u) {
  const int lane = threadIdx.x & 31, d = kGroup * u.group + lane, half = A.half;
  const __nv_bfloat16* x = A.k + u.t * A.k_stride + (int64_t)u.head * D;
  // the value's partner in the rotation, if it is turned
  const bool is_turned = d < 2 * half, second = A.inter ? (d & 1) != 0 : d >= half;
  const int j = A.inter ? d >> 1 : second ? d - half : d, other = !is_turned ? d : A.inter ? d ^ 1 : second ? j : d + half;
  float y = __bfloat162float(x[d]), z = __bfloat162float(x[other]);
  if (A.k_weight) {
    auto weight = [&](int e) {
      return __fadd_rn(A.weight_f32 ? static_cast<const float*>(A.k_weight)[e]
                                    : __bfloat162float(static_cast<const __nv_bfloat16*>(A.k_weight)[e]), A.w0);
    };
    const float wy = weight(d), wz = weight(other);
    float v[D / 32];
#pragma unroll
    for (int e = 0; e < D / 32; ++e) v[e] = __bfloat162float(x[lane + 32 * e]);
    Two ss{0.f, 0.f};
#pragma unroll
    for (int e = 0; e < D / 32; ++e) {  // squares of 8 bits are exact
      const Two s = two_sum(ss.hi, product(v[e], v[e]));
      ss = Two{s.hi, ss.lo + s.lo};
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
      ss = ss + Two{__shfl_xor_sync(0xffffffffu, ss.hi, o), __shfl_xor_sync(0xffffffffu, ss.lo, o)};
    const float r = rsqrtf(__fadd_rn(ss.hi * (1.f / D), A.eps));
    y = product(product(y, r), wy);
    z = product(product(z, r), wz);
  }
  if (is_turned) {
    Two c, s;
    cos_sin_turns((uint64_t)u.pos * freq[j], c, s);
    const float yc = product(y, c.hi), zs = product(z, s.hi);
    y = second ? __fadd_rn(yc, zs) : __fsub_rn(yc, zs);
  }
  float top = fabsf(y);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
  const uint32_t bits = five_bits(__fdiv_rn(top, 7.f));
  const int n = bits ? (int)floorf(__fadd_rn(__fdiv_rn(fabsf(y), __uint_as_float(bits)), 0.5f)) : 0;
  const int code = 8 + (y < 0.f ? -n : n), pair = code | __shfl_down_sync(0xffffffffu, code, 1) << 4;
  if ((lane & 1) == 0) static_cast<uint8_t*>(A.kv.k)[u.row * (D / 2) + d / 2] = (uint8_t)pair;
  if (lane == 0) A.kv.ks[u.row * (D / kGroup) + u.group] = __ushort_as_bfloat16((unsigned short)(bits >> 16));
}

template <int D, int BITS, int CAP>
__global__ void __launch_bounds__(kThreads, 2) append_kernel(const __grid_constant__ AppendArgs A,
                                                             const __grid_constant__ SegTable<CAP> seg) {
  constexpr int G = D / 16, S = 32 / G;
  extern __shared__ uint4 dynamic[];
  AppendShared<D, BITS>& sh = *reinterpret_cast<AppendShared<D, BITS>*>(dynamic);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, slot = lane / G, i = lane % G;
  const LaneMap m = lane_map<D>(i, A.half, A.inter);
  // a lane's two vectors of a value head: 16 consecutive values in 4 bits, else as its neighbours'
  const int va = BITS == 4 ? 16 * i : 8 * i, vb = BITS == 4 ? 16 * i + 8 : D / 2 + 8 * i;
  const bool norm = A.q_weight != nullptr;
  const int Hkv = A.kv.Hkv, nq = (A.Hq + S - 1) / S, nk = (Hkv + S - 1) / S, steps = nq + 2 * nk;
  // block rows (blockIdx.y) share a row's steps
  const int begin = steps * (int)blockIdx.y / (int)gridDim.y, end = steps * ((int)blockIdx.y + 1) / (int)gridDim.y;
  const int64_t first = (int64_t)blockIdx.x * kWarps + warp, stride = (int64_t)gridDim.x * kWarps;

  // the copies' place in the walk: x is the lane's first vector of the head, the second lies dx behind
  int64_t at = first;
  int s_at = begin, h_at = 0, heads_at = 0, dx = 0;
  const __nv_bfloat16* x = nullptr;
  auto place_copies = [&]() {
    const int part = s_at < nq ? 0 : s_at < nq + nk ? 1 : 2;
    h_at = slot + (s_at - (part == 0 ? 0 : part == 1 ? nq : nq + nk)) * S;
    heads_at = part == 0 ? A.Hq : Hkv;
    dx = part == 2 ? vb - va : m.b - m.a;
    x = (part == 0 ? A.q + at * A.q_stride : part == 1 ? A.k + at * A.k_stride : A.v + at * A.v_stride) + h_at * D +
        (part == 2 ? va : m.a);
  };
  place_copies();
  cudaGridDependencySynchronize();
  auto fetch = [&](int stage) {
    if (at < A.T) {
      if (h_at < heads_at) {
        copy16(&sh.ring[stage][0][threadIdx.x], x);
        copy16(&sh.ring[stage][1][threadIdx.x], x + dx);
      }
      h_at += S;
      x += S * D;
      ++s_at;
      if (s_at == end) {
        s_at = begin;
        at += stride;
        if (at < A.T) place_copies();
      } else if (s_at == nq || s_at == nq + nk) {
        place_copies();
      }
    }
    copies_commit();
  };
#pragma unroll
  for (int k = 0; k < kDepth - 1; ++k) fetch(k);
  for (int j = threadIdx.x; j < A.half; j += kThreads) sh.freq[j] = turn_fraction(A.inv_freq[j]);
  if (norm) {
    for (int d = threadIdx.x; d < 2 * D; d += kThreads) {
      const void* w = d < D ? A.q_weight : A.k_weight;
      const int e = d % D;
      sh.w[d / D][split_at(e, D)] = A.w0 + (A.weight_f32 ? static_cast<const float*>(w)[e]
                                                     : __bfloat162float(static_cast<const __nv_bfloat16*>(w)[e]));
    }
  }
  __syncthreads();

  int stage = 0;
  Place coming = place_of(stream_of(seg, A.lens, A.starts, first, A.T), A.by_ps, seg, A.table, A.max_pages, first, A.T);
  StreamOf after = stream_of(seg, A.lens, A.starts, first + stride, A.T);
  for (int64_t t = first; t < A.T; t += stride) {
    const Place at_row = coming;
    coming = place_of(after, A.by_ps, seg, A.table, A.max_pages, t + stride, A.T);
    after = stream_of(seg, A.lens, A.starts, t + 2 * stride, A.T);
    const bool stored = has_page(A.kv, at_row, A.status);
    const Angles ang = row_angles((int)at_row.pos, sh.freq, A.half, sh.cs[warp], sh.sn[warp], lane, m, A.inter);
    auto next = [&](uint4& ra, uint4& rb) {
      fetch(stage == 0 ? kDepth - 1 : stage - 1);
      copies_wait<kDepth - 1>();
      ra = sh.ring[stage][0][threadIdx.x];
      rb = sh.ring[stage][1][threadIdx.x];
      stage = stage == kDepth - 1 ? 0 : stage + 1;
    };
    // norm and rotation of the head in the next step
    auto turned = [&](const float* w, Vec8& a, Vec8& b) {
      uint4 ra, rb;
      next(ra, rb);
      a = unpack8(ra);
      b = unpack8(rb);
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
      turn(a, b, ang, m, A.inter);
    };
    Vec8 a, b;
    {
      int h = slot + begin * S;
      __nv_bfloat16* y = A.q_out + (t * A.Hq + h) * D + m.a;
      for (int step = begin; step < min(end, nq); ++step, h += S, y += S * D) {
        turned(sh.w[0], a, b);
        if (h < A.Hq) {
          *reinterpret_cast<uint4*>(y) = pack8(a);
          *reinterpret_cast<uint4*>(y + m.b - m.a) = pack8(b);
        }
      }
    }
    const int64_t page_row = cache_row(A.kv, at_row.entry, 0, at_row.slot);
    for (int step = max(begin, nq); step < min(end, nq + nk); ++step) {
      const int h = slot + (step - nq) * S;
      const bool live = h < Hkv && stored;
      const int64_t row = page_row + (int64_t)h * A.kv.ps;
      turned(sh.w[1], a, b);
      if constexpr (BITS == 16) {
        if (live) {
          __nv_bfloat16* y = static_cast<__nv_bfloat16*>(A.kv.k) + row * D + m.a;
          *reinterpret_cast<uint4*>(y) = pack8(a);
          *reinterpret_cast<uint4*>(y + m.b - m.a) = pack8(b);
        }
      } else {  // groups of 32 lie across lanes: through shared memory into the values' order
        float* keys = sh.k[warp];
        store8(a, keys, slot * D + m.a);
        store8(b, keys, slot * D + m.b);
        const float around = magnitude3(magnitude8(a), magnitude8(b), 0.f);
        sh.size[warp][(slot * D + m.a) / 8] = norm || (m.ta && at_row.pos) ? around : 0.f;
        sh.size[warp][(slot * D + m.b) / 8] = norm || (m.tb && at_row.pos) ? around : 0.f;
        __syncwarp();
        Vec8 v[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) v[e] = load8(keys + spread(16 * lane + 8 * e), keys + spread(16 * lane + 8 * e + 4));
        const float2 sizes = *reinterpret_cast<const float2*>(&sh.size[warp][2 * lane]);
        __syncwarp();
        __nv_bfloat16 scale;
        bool near;
        const uint2 c = quantise16<true>(v, magnitude3(sizes.x, sizes.y, sizes.x), scale, near);
        uint32_t again = __ballot_sync(0xffffffffu, near && live);  // lanes; a group's first one stands for it
        again = (again | again >> 1) & 0x55555555u;
        if (live && !(again >> (lane & ~1) & 1)) store_codes<D>(c, scale, A.kv.k, A.kv.ks, row, i);
        for (; again; again &= again - 1) {
          const int from = __ffs(again) - 1, head = from / G + (step - nq) * S;
          settle_group<D>(A, sh.freq, Undecided{page_row + (int64_t)head * A.kv.ps, (int)t, head, from % G / 2, at_row.pos});
        }
      }
    }
    for (int step = max(begin, nq + nk); step < end; ++step) {
      const int h = slot + (step - nq - nk) * S;
      const bool live = h < Hkv && stored;
      const int64_t row = page_row + (int64_t)h * A.kv.ps;
      uint4 ra, rb;
      next(ra, rb);
      if constexpr (BITS == 16) {
        if (live) {
          __nv_bfloat16* y = static_cast<__nv_bfloat16*>(A.kv.v) + row * D;
          *reinterpret_cast<uint4*>(y + va) = ra;
          *reinterpret_cast<uint4*>(y + vb) = rb;
        }
      } else {
        Vec8 v[2] = {unpack8(ra), unpack8(rb)};
        __nv_bfloat16 scale;
        bool near;
        const uint2 c = quantise16<false>(v, 0.f, scale, near);
        if (live) store_codes<D>(c, scale, A.kv.v, A.kv.vs, row, i);
      }
    }
  }
}

// A warp takes a row: first its keys, then its values, 8 values a lane and step.
template <int D, int BITS, int CAP>
__global__ void __launch_bounds__(kThreads) read_kernel(const ReadArgs A, const __grid_constant__ SegTable<CAP> seg) {
  constexpr int V = D / 8;  // vectors of a head
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t t = (int64_t)blockIdx.x * kWarps + warp;
  if (t >= A.T) return;
  cudaGridDependencySynchronize();
  const Place at = place_of(stream_of(seg, A.lens, nullptr, t, A.T), A.by_ps, seg, A.table, A.max_pages, t, A.T);
  const bool stored = has_page(A.kv, at, A.status);
  const int n = A.kv.Hkv * V;
  uint4* out[2] = {reinterpret_cast<uint4*>(A.k_out) + t * n, reinterpret_cast<uint4*>(A.v_out) + t * n};
  // keys and values, two vectors of each at once on their way
  const int64_t row0 = cache_row(A.kv, at.entry, 0, at.slot);
  constexpr int BATCH = 2;
  for (int u0 = lane; u0 < n; u0 += 32 * BATCH) {
    uint4 y[BATCH][2];
    uint32_t w[BATCH][2];
    __nv_bfloat16 sc[BATCH][2];
#pragma unroll
    for (int k = 0; k < BATCH; ++k)
#pragma unroll
      for (int which = 0; which < 2; ++which) {
        const int u = u0 + 32 * k;
        const void* pool = which ? A.kv.v : A.kv.k;
        const int64_t row = row0 + (int64_t)(u / V) * A.kv.ps;
        y[k][which] = make_uint4(0, 0, 0, 0);
        w[k][which] = 0;
        sc[k][which] = __ushort_as_bfloat16(0);
        if (stored && u < n) {
          if (BITS == 16) {
            y[k][which] = static_cast<const uint4*>(pool)[row * V + u % V];
          } else {
            w[k][which] = static_cast<const uint32_t*>(pool)[row * V + u % V];
            sc[k][which] = (which ? A.kv.vs : A.kv.ks)[row * (D / kGroup) + u % V / 4];
          }
        }
      }
#pragma unroll
    for (int k = 0; k < BATCH; ++k)
#pragma unroll
      for (int which = 0; which < 2; ++which) {
        const int u = u0 + 32 * k;
        if (BITS == 4) {
          const __nv_bfloat162 s2 = __bfloat162bfloat162(sc[k][which]);
          const uint4 p = decode8(w[k][which], s2, __hmul2(s2, __float2bfloat162_rn(-24.f)));
          y[k][which] = make_uint4(__byte_perm(p.x, p.y, 0x5410), __byte_perm(p.z, p.w, 0x5410),
                                   __byte_perm(p.x, p.y, 0x7632), __byte_perm(p.z, p.w, 0x7632));
        }
        if (u < n) out[which][u] = y[k][which];
      }
  }
}

template <int D, int BITS, int CAP>
cudaError_t append_c(const AppendArgs& a, int S, const int32_t* off, cudaStream_t st) {
  const SegTable<CAP> seg = make_segs<CAP>(0, S, off);
  constexpr int smem = (int)sizeof(AppendShared<D, BITS>);
  const cudaError_t e = allow_shared<&append_kernel<D, BITS, CAP>>(a.device, smem);
  if (e != cudaSuccess) return e;
  const int heads = 512 / D, steps = (a.Hq + heads - 1) / heads + 2 * ((a.kv.Hkv + heads - 1) / heads);
  // few rows share their steps among block rows; from two resident blocks per SM on a warp takes several rows (a block
  // needs some 2.5 us before its first), up to six rounds of blocks where there are more than 8 rows for each warp
  const int64_t need = (a.T + kWarps - 1) / kWarps, spare = kResident / need;
  int64_t rounds = need / (8 * kResident);
  rounds = rounds < 1 ? 1 : rounds > 6 ? 6 : rounds;
  const int64_t blocks = need <= kResident ? need : rounds * kResident;
  const dim3 grid((unsigned)blocks, (unsigned)(spare < 1 ? 1 : spare < steps ? spare : steps));
  return launch_behind_shared(append_kernel<D, BITS, CAP>, grid, dim3(kThreads), smem, st, a, seg);
}

template <int D, int BITS, int CAP>
cudaError_t read_c(const ReadArgs& a, int S, const int32_t* off, cudaStream_t st) {
  const SegTable<CAP> seg = make_segs<CAP>(0, S, off);
  return launch_behind(read_kernel<D, BITS, CAP>, dim3((unsigned)((a.T + kWarps - 1) / kWarps)), dim3(kThreads), st, a, seg);
}

template <int D, int CAP>
cudaError_t append_d(const AppendArgs& a, int S, const int32_t* off, cudaStream_t st) {
  return a.kv.ks ? append_c<D, 4, CAP>(a, S, off, st) : append_c<D, 16, CAP>(a, S, off, st);
}
template <int D, int CAP>
cudaError_t read_d(const ReadArgs& a, int S, const int32_t* off, cudaStream_t st) {
  return a.kv.ks ? read_c<D, 4, CAP>(a, S, off, st) : read_c<D, 16, CAP>(a, S, off, st);
}

}  // namespace

cudaError_t launch_append(int D, const AppendArgs& a, int S, const int32_t* off, cudaStream_t st) {
  if (a.T <= 0) return cudaSuccess;
  const bool few = S <= kSmallSegs;
  switch (D) {
    case 64:
      return few ? append_d<64, kSmallSegs>(a, S, off, st) : append_d<64, kMaxSegs>(a, S, off, st);
    case 128:
      return few ? append_d<128, kSmallSegs>(a, S, off, st) : append_d<128, kMaxSegs>(a, S, off, st);
    case 512:
      return few ? append_d<512, kSmallSegs>(a, S, off, st) : append_d<512, kMaxSegs>(a, S, off, st);
    default:
      return cudaErrorInvalidValue;
  }
}

cudaError_t launch_read(int D, const ReadArgs& a, int S, const int32_t* off, cudaStream_t st) {
  if (a.T <= 0) return cudaSuccess;
  const bool few = S <= kSmallSegs;
  switch (D) {
    case 64:
      return few ? read_d<64, kSmallSegs>(a, S, off, st) : read_d<64, kMaxSegs>(a, S, off, st);
    case 128:
      return few ? read_d<128, kSmallSegs>(a, S, off, st) : read_d<128, kMaxSegs>(a, S, off, st);
    case 512:
      return few ? read_d<512, kSmallSegs>(a, S, off, st) : read_d<512, kMaxSegs>(a, S, off, st);
    default:
      return cudaErrorInvalidValue;
  }
}

}  // namespace dkv
