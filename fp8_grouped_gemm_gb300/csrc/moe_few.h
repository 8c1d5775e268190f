// Shared by the two forms of the expert layer for a few tokens.
#pragma once
#include "mgq_internal.h"

namespace mgq {

// block scaling of the operands
enum { kMX = 0, kNV = 1, kBLK = 2, kTEN = 3 };

// The form for at most kSmallT tokens (moe_few_small.cu); `ws` has
// few_small_workspace() bytes, 256-byte aligned. Arguments are checked.
constexpr int kSmallT = 8;
size_t few_small_workspace(int T, int k, int64_t F, int kind);
int few_small_forward(int kind, const void* x, int T, int64_t H, int64_t F, const int32_t* idx, const float* probs, int k,
                      int E, const mgq_operand* W1, const mgq_operand* W2, const float* x_scale, const float* h_scale,
                      void* out, uint8_t* ws, cudaStream_t s);


// Whether a call takes that form: few tokens, and weights of the experts they
// can pick so small that its two launches beat the line's four. The line
// streams at the memory's rate but starts and joins for about 14 us; the small
// form needs 6 us and reads at about 2.5 TB/s (its conversions bound it: MX
// scales every 32 elements, NVFP4 converts to f16). Measured, small / line:
//   per tensor  38 MB 13.3 / 19.4 us,  75 MB 23.3 / 27.4,  100 MB 33.1 / 27.5
//   1x128       38 MB 15.0 / 21.2 us,  75 MB 27.2 / 28.9,  151 MB 45.5 / 42.2
//   MXFP8       26 MB 15.5 / 18.7 us,  39 MB 18.5 / 19.5,   52 MB 25.7 / 23.6
//   NVFP4       14 MB 12.7 / 16.5 us,  21 MB 13.5 / 19.1,   28 MB 23.9 / 18.9
inline bool few_is_small(int kind, int T, int k, int E, int64_t H, int64_t F) {
  const int64_t experts = static_cast<int64_t>(T) * k < E ? static_cast<int64_t>(T) * k : E;
  const int64_t bytes = experts * 3 * H * F * (kind == kNV ? 9 : 16) / 16;
  return T <= kSmallT && bytes <= (kind == kNV ? 24 : kind == kMX ? 40 : 72) * int64_t(1000000);
}

}  // namespace mgq
