// kv_layout.h -- the paged FP4 key/value cache (layout defined in
// include/fp4q.h) as its kernels address it.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "fp4q_internal.h"

namespace fp4q {

// FMT: FP4Q_NVFP4 or FP4Q_MXFP4; D: head dimension.
template <int FMT, int D>
struct KvLayout {
  static constexpr int BLK = FMT == FP4Q_NVFP4 ? 16 : 32;
  static constexpr int SB = D / BLK;  // scale bytes of a token (K or V)
  static constexpr int J = D / 32;    // 32-element runs of a token
  // Bytes of one (page, head): K codes, V codes, K scales, V scales.
  __host__ __device__ static constexpr int bytes(int page) { return page * (D + 2 * SB); }
  __host__ __device__ static constexpr int k_codes(int) { return 0; }
  __host__ __device__ static constexpr int v_codes(int page) { return page * (D / 2); }
  __host__ __device__ static constexpr int k_scales(int page) { return page * D; }
  __host__ __device__ static constexpr int v_scales(int page) { return page * (D + SB); }
};

// Sequence of new-token row r: the last b with offsets[b] <= r (sequences
// without new tokens are passed over); r in [0, offsets[B]).
__device__ __forceinline__ int kv_sequence(const int32_t* off, int B, int64_t r) {
  int lo = 0, hi = B;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (off[mid] <= r) lo = mid;
    else hi = mid;
  }
  return lo;
}

}  // namespace fp4q
