// kernels.h -- launch interface between the C-ABI layer (api.cu) and the kernels.
#pragma once
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "plan.h"

namespace dkv {

// Limit of every bounded wait in a normal launch (a healthy wait ends in microseconds).
constexpr uint64_t kLaunchWaitLimitNs = 2000000000ull;

struct FwdArgs {
  const QTileItem* items;
  __nv_bfloat16* out;
  float* lse;
  int T, Hq, Hkv, window;
  float scale_log2;  // softmax scale * log2(e)
  uint32_t* status;
  uint64_t wait_limit_ns = kLaunchWaitLimitNs;
  // failure-path self-test only (-1 otherwise): the K/V ring unit with this index is
  // never loaded, so the wait for it runs out after wait_limit_ns
  int test_skip_unit = -1;
};

// Query tile rows / key tile size of the forward kernel for head dimension D.
int fwd_query_tile(int D);
int fwd_key_tile(int D);
cudaError_t launch_fwd(int D, const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv, const FwdArgs& a,
                       int n_items, cudaStream_t st);

struct PrepArgs {
  const __nv_bfloat16* out;
  const __nv_bfloat16* dout;
  const float* lse;
  float* delta;  // [Hq, T]
  float* lse2;   // [Hq, T], lse * log2(e)
  int64_t T;
  int Hq, D;
  int h_lo = 0, h_hi = -1;  // q-heads [h_lo, h_hi) are prepared (h_hi < 0: all)
  // the dQ work list to check (and to empty any entry outside the tensors) before the
  // dQ kernel runs; null: none
  QTileItem* check_items = nullptr;
  int n_check = 0, check_tile = 128;
  uint32_t* status = nullptr;
};
cudaError_t launch_prep(const PrepArgs& a, cudaStream_t st);

struct DqArgs {
  const QTileItem* items;
  const float* delta;
  const float* lse2;
  __nv_bfloat16* dq;
  int T, Hq, Hkv, window;
  float scale_log2;  // softmax scale * log2(e)
  float scale;       // softmax scale
  uint32_t* status;
  int n_items = 0;   // set by launch_dq
};
int dq_query_tile(int D);
int dq_key_tile(int D);
cudaError_t launch_dq(int D, const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv,
                      const CUtensorMap& tdo, const DqArgs& a, int n_items, cudaStream_t st);

struct DkvArgs {
  const KVTileItem* items;
  const QBlock* qblocks;
  const float* delta;
  const float* lse2;
  __nv_bfloat16* dk;
  __nv_bfloat16* dv;
  float* partial;  // [slot][2][key_tile][D] fp32
  int T, Hq, Hkv, window;
  float scale_log2;
  float scale;
  uint32_t* status;
  int nslots = 0;  // partial slots in `partial` (work items naming another slot are out of range)
  uint64_t wait_limit_ns = kLaunchWaitLimitNs;
  // failure-path self-test only (-1 otherwise): the Q/dO block of this iteration of
  // the first work item gets one arrival too few, so the wait for it runs out
  int test_skip_iter = -1;
};
int dkv_key_tile(int D);
int dkv_query_block(int D);
cudaError_t launch_dkv(int D, const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv,
                       const CUtensorMap& tdo, const DkvArgs& a, int n_items, cudaStream_t st);

struct ReduceArgs {
  const ReduceItem* items;
  const float* partial;
  __nv_bfloat16* dk;
  __nv_bfloat16* dv;
  int Hkv, D, key_tile;
  int64_t T = 0;        // rows of dk / dv
  int total_slots = 0;  // partial slots in `partial`
  uint32_t* status = nullptr;
};
cudaError_t launch_reduce(const ReduceArgs& a, int n_items, cudaStream_t st);

// ---- head dimension 512 backward (bwd512.cu)
struct PdsArgs {
  const QTileItem* items;
  const int32_t* block_base;
  const float* lse2;
  const float* delta;
  __nv_bfloat16* p_out;   // P blocks (written)
  __nv_bfloat16* ds_out;  // dS blocks (written)
  int T, Hq, Hkv, window;
  float scale_log2;
  uint32_t* status;
  int64_t n_blocks = 0;  // blocks in p_out and ds_out
  uint64_t wait_limit_ns = kLaunchWaitLimitNs;
  // failure-path self-test only (-1 otherwise): the K/V ring unit with this index is
  // never loaded, so the wait for it runs out after wait_limit_ns
  int test_skip_unit = -1;
};
// Both blocks of every (query tile, key tile) pair in one pass: P = exp(S - LSE)
// into a.p_out and dS = P (dP - Delta) into a.ds_out.
cudaError_t launch_pds_fused(const CUtensorMap& tq, const CUtensorMap& tdo, const CUtensorMap& tk,
                             const CUtensorMap& tv, const PdsArgs& a, int n_items, cudaStream_t st);

struct XtgArgs {
  const XTItem* items;
  const XTEntry* entries;
  __nv_bfloat16* out;  // dV or dK [T, Hkv, 512]
  float* partial;      // [slot][2][128][512]
  int region;          // partial half: 0 = dK, 1 = dV
  int T, Hq, Hkv;
  float mul;
  uint32_t* status;
  int64_t n_entries = 0;  // entries in `entries`
  int64_t n_blocks = 0;   // P / dS blocks the entries may name
  int nslots = 0;         // partial slots in `partial`
};
cudaError_t launch_xtg(const CUtensorMap& tBlk, const CUtensorMap& tB, const XtgArgs& a, int n_items, cudaStream_t st);

struct Dq512Args {
  const QTileItem* items;
  const int32_t* block_base;
  __nv_bfloat16* dq;
  int T, Hq, Hkv;
  float scale;
  uint32_t* status;
  int64_t n_blocks = 0;  // dS blocks
};
cudaError_t launch_dq512(const CUtensorMap& tBlk, const CUtensorMap& tK, const Dq512Args& a, int n_items,
                         cudaStream_t st);

// One CTA waits on an mbarrier that nothing completes, with a bounded wait of limit_ns.
cudaError_t launch_selftest_timeout(uint64_t limit_ns, uint32_t* status, cudaStream_t st);

// ---- per-token tensors between the replicated and the packed layout (pack.cu)
// kind 0 = pack (replicated -> packed), 1 = unpack (packed -> replicated),
// 2 = fold (replicated -> packed, prompt rows summed over the replicas).
// Rows are row_elems bf16 (a multiple of 8); d_off is R_offsets in device memory.
int pack_group_lanes(int row_elems);
cudaError_t launch_pack(int kind, const void* src, void* dst, const int32_t* d_off, int P, int N, int64_t T,
                        int row_elems, int num_sms, cudaStream_t st);

// ---- per-head norm and rotation of q and k (rope.cu)
struct RopeArgs {
  const __nv_bfloat16 *q, *k;            // projections' rows, head h of row t at t * stride + h * D
  int64_t q_stride, k_stride;            // elements
  const __nv_bfloat16 *dq_out, *dk_out;  // backward: gradients of the rotated q and k, contiguous
  __nv_bfloat16 *q_out, *k_out;          // written: rotated q and k, or (backward) the gradients of q and k
  int64_t q_out_stride, k_out_stride;
  const void *q_weight, *k_weight;       // D values each; both null: no norm
  const float* inv_freq;                 // half values
  float* partial;                        // backward: [block][D] weight gradients, q's blocks first
  int64_t T;
  int Hq, Hkv, half;                     // half = rope_dim / 2
  float w0, eps;
  bool weight_f32, inter;
};
// One launch over all rows; the backward adds a second one that sums the weight gradients.
cudaError_t launch_rope(bool backward, int D, const RopeArgs& a, int P, int N, const int32_t* off, float* dqw,
                        float* dkw, cudaStream_t st);
size_t rope_workspace_bytes(int64_t T, int Hq, int Hkv, int D);

// ---- token log-probabilities (logprobs.cu)
struct LogpArgs {
  const void* logits;       // bf16 or fp32 rows of V values, `stride` elements apart
  int64_t stride;
  int V;
  float scale;
  const int64_t* tokens;    // response tokens in packed order; < 0: ignored
  float *logp, *entropy, *lse;  // forward: written (entropy, lse may be null); backward: entropy, lse read
  const float *dlogp, *dentropy;
  void* dlogits;
  int64_t dstride;
  uint32_t* status;
};
cudaError_t launch_logprobs(bool backward, bool f32, const LogpArgs& a, int P, int N, const int32_t* off,
                            cudaStream_t st);

// ---- clipped policy loss (policy.cu)
constexpr int kPolicyChunk = 1024;  // response tokens of one block

// An fp64 value as the sum of two fp32 values.
struct Bound {
  float hi, lo;
};
struct PolicyArgs {
  const float *logp, *old_logp, *ref_logp, *entropy, *adv;  // ref_logp, entropy may be null
  const uint8_t* mask;                                      // null: every token is live
  int per_token, reduction, has_dual;
  Bound up, down, dual;              // the bounds on the ratio, as differences of log-probabilities
  Bound add_up, add_down, add_dual;  // and as the ratio less 1
  double kl_coef, entropy_coef;
  float *loss, *stats, *weights;  // forward: written; backward: weights read
  void* records;
  const float* dloss;
  float *dlogp, *dentropy;
};
// Forward: the sums and a second launch of one block that joins them.  Backward: one launch.
cudaError_t launch_policy(bool backward, const PolicyArgs& a, int N, const int32_t* off, cudaStream_t st);
size_t policy_workspace_bytes(int N, const int32_t* off);

// Quotients of 0 <= x < 2^31 by a d that the host knows: with 2^s the first power of two from d on,
// x / d = (x + floor(x m / 2^32)) / 2^s for m = floor(2^32 (2^s - d) / d) + 1 (Granlund and Montgomery).
struct FastDiv {
  uint32_t d, mul, shift;
  FastDiv(int by = 1) : d((uint32_t)by), mul(0), shift(0) {
    while ((1u << shift) < d) ++shift;
    mul = (uint32_t)((((uint64_t)1 << 32) * ((((uint64_t)1) << shift) - d)) / d + 1);
  }
#ifdef __CUDACC__
  __device__ __forceinline__ int operator()(int x) const {
    return (int)((__umulhi((uint32_t)x, mul) + (uint32_t)x) >> shift);
  }
#endif
};
// ---- paged key/value cache (cache.cu)
struct PagedKV {
  void *k, *v;              // [pages, Hkv, ps, D] bf16, or codes [pages, Hkv, ps, D / 2]
  __nv_bfloat16 *ks, *vs;   // scales [pages, Hkv, ps, D / 32] of the codes; null: bf16
  int pages, ps, Hkv;
};
struct AppendArgs {
  const __nv_bfloat16 *q, *k, *v;       // rows, head h of row t at t * stride + h * D
  int64_t q_stride, k_stride, v_stride;  // elements
  __nv_bfloat16* q_out;                  // contiguous
  const void *q_weight, *k_weight;       // D values each; both null: no norm
  const float* inv_freq;                 // half values
  PagedKV kv;
  const int32_t *table, *lens, *starts;  // [streams, max_pages], [streams], [streams]
  int max_pages;
  int64_t T;
  int Hq, half;
  float w0, eps;
  bool weight_f32, inter;
  FastDiv by_ps;
  uint32_t* status;
  int device;
};
cudaError_t launch_append(int D, const AppendArgs& a, int S, const int32_t* off, cudaStream_t st);

struct ReadArgs {
  PagedKV kv;
  const int32_t *table, *lens;
  int max_pages;
  int64_t T;
  __nv_bfloat16 *k_out, *v_out;  // contiguous
  FastDiv by_ps;
  uint32_t* status;
};
cudaError_t launch_read(int D, const ReadArgs& a, int S, const int32_t* off, cudaStream_t st);

// ---- attention of one token per response over the cache (decode.cu)
constexpr int kMaxResponses = 8192;

struct DecodeArgs {
  const __nv_bfloat16* q;  // head h of response b at b * q_stride + h * D
  int64_t q_stride;        // elements
  PagedKV kv;
  const int32_t *prompt_table, *prompt_lens;  // [G, max_prompt_pages], [G]; null: no prompts
  const int32_t *table, *lens;                // [B, max_pages], [B]
  int max_prompt_pages, max_pages;
  int G, B, Hq, window;
  float scale_log2;  // softmax scale * log2(e)
  __nv_bfloat16* out;
  float* lse;        // may be null
  void* workspace;
  uint32_t* status;
  FastDiv by_ps, by_heads;  // by the page size and by Hq / Hkv
  int device;
  bool big;          // launch_prompt's kernel runs before and takes the prompts that are worth it
  uint64_t wait_limit_ns = kLaunchWaitLimitNs;
  // failure-path self-test only (-1 otherwise): the tile of keys with this index in each block of launch_prompt's kernel
  // is never loaded, so the wait for it runs out after wait_limit_ns
  int test_skip_tile = -1;
};
// Prompts of groups with this many rows and more go to launch_prompt's kernel ...
constexpr int kBigRows = 32;
// ... where the tokens that the groups see times their rows and the kv-heads come to this much.  32 responses, 8 kv-heads
// of 128 with 4 rows each, behind 1,500 / 2,500 / 3,400 tokens (1.5, 2.6, 3.5 M): 24 / 24 / 26 us there, 23 / 29 / 35 by
// decode_walk.cuh's warps alone in bf16; 22 / 23 / 23 and 17 / 22 / 26 in 4 bits.  Heads of 64, bf16: 19 and 17 at 2.3 M,
// 20 and 23 at 3.8 M.
__host__ __device__ inline unsigned long long big_work(const PagedKV& kv) { return kv.ks ? 3400000 : 2400000; }
constexpr int kBigGroups = 512;      // most groups of a call with that kernel: their lengths are in shared memory
constexpr int kBigResponses = 4096;  // and most responses
// tk, tv: views (make_tmap, boxes of 16 rows) of the bf16 pools, used where a.big and the cache holds bf16
cudaError_t launch_decode(int D, const DecodeArgs& a, const CUtensorMap& tk, const CUtensorMap& tv, const int32_t* groups,
                          cudaStream_t st);
cudaError_t launch_walk_window(int D, const DecodeArgs& a, const int32_t* groups, cudaStream_t st);
cudaError_t launch_prompt(int D, const DecodeArgs& a, const CUtensorMap& tk, const CUtensorMap& tv, const int32_t* groups,
                          cudaStream_t st);
size_t decode_workspace_bytes(int B, int Hq, int Hkv, int D);

}  // namespace dkv
