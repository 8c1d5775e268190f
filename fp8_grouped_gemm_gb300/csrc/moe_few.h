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

// Whether a call takes that form. Its two launches start in less time than the
// line's four, but a warp of it works through its stretch of H one 128-element
// unit after another, so its time grows with H and, past one wave of its
// first launch, with the ffn rows of the experts that the call can pick. The
// line is near the memory's rate at any size and needs 11 to 16 us to start and
// to join. Measured at (E, k, H, F) and T tokens, small / line, microseconds:
//   rows   per tensor                       1x128
//   4096   (16, 2, 1024, 1024) T2  8.3/11.9  9.4/14.5
//   8192   (16, 2, 4096, 1024) T4 19.9/23.3 22.9/26.6
//   9216   (64, 6, 2048, 1536) T1 16.5/18.8 21.4/22.3
//  12288  (128, 8, 2048,  768) T2 23.0/23.1 27.5/25.1
//  12288   (32, 4, 1024, 1024) T3 16.7/13.4 20.0/15.8
//   1024   (32, 2, 8192,  512) T1 20.8/14.7 26.5/16.6
//   rows   NVFP4 (conversions to f16)
//   4096   (16, 2, 4096, 1024) T2 11.7/15.7
//   6144  (128, 8, 2048,  768) T1 12.0/14.3
//   6144   (16, 2, 4096, 1024) T3 17.4/16.9
//   8192   (16, 2, 1024, 1024) T4 10.5/12.2
//   9216   (64, 6, 2048, 1536) T1 15.1/15.2
//  12288   (16, 2,  512, 2048) T3 13.7/12.5
//   1024   (32, 2, 8192,  512) T1 16.9/15.4
//   rows   MXFP8 (a scale every 32 elements: twice the work of a unit)
//   4096   (32, 4, 1024, 1024) T1 10.4/12.9
//   6144   (32, 4, 1024,  512) T3 13.3/12.1
//   8192   (16, 2, 1024, 1024) T4 14.2/13.4
//   1024   (32, 2, 2048,  512) T1 13.2/12.5
inline bool few_is_small(int kind, int T, int k, int E, int64_t H, int64_t F) {
  const int64_t experts = static_cast<int64_t>(T) * k < E ? static_cast<int64_t>(T) * k : E;
  // 9728: one wave of 32-row CTAs, two on an SM (NVFP4: of 16-row CTAs, four on an SM)
  const int64_t rows = kind == kMX || (kind == kNV && H > 2048) ? 4864 : 9728;
  return T <= kSmallT && H <= (kind == kMX ? 1024 : 4096) && experts * F <= rows;
}

}  // namespace mgq
