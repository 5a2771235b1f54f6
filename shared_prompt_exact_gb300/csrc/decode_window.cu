// decode_window.cu -- the warps' part of dualkv_decode under a sliding window.
#include "decode_walk.cuh"

namespace dkv {

cudaError_t launch_walk_window(int D, const DecodeArgs& a, const int32_t* groups, cudaStream_t st) {
  return walk<true>(D, a, groups, st);
}

}  // namespace dkv
