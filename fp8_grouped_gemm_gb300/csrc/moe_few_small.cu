// The expert layer for at most eight tokens: the smallest decode calls, where
// latency counts as much as bandwidth (definition and entry point: moe_few.cu).
//
// An expert then has at most eight rows, one N = 8 tile of the warp-level
// tensor-core instruction, which takes the weights' codes from registers as
// they come from memory: no ring, no tensor memory, no partial sums between
// CTAs. Two launches, the second started while the first drains; its weights
// are requested before it waits for the first.
//   small_gateup_kernel   a CTA: 32 gate and 32 up rows of one expert (NVFP4: 16
//                         and 16, one block of its scales); its warps split the
//                         contraction and quantise their stretch of the tokens'
//                         x on the way; SwiGLU, h quantised
//   small_down_kernel     a CTA: 16 rows of W2 of every picked expert, its warps
//                         split all of their contractions; out
// All sums run in an order that only the sizes and the routing decide. An expert
// that a token names more than once is one row, with the sum of its
// probabilities: so an expert has at most as many rows as there are tokens.
//
// Bound by latency: the launch, the ids, then a warp's units one after another
// (gate and up: a unit's loads together, the next unit's behind its products;
// down: four units' loads together) and the reduction over the warps. Measured:
// one token, 2 experts of (1024, 1024), per tensor 5.9 us, NVFP4 6.5, 1x128 7.0,
// MXFP8 7.4; one token, 8 experts of (2048, 768): per tensor 13.4 us, 2.8 TB/s,
// NVFP4 12.1 us, 1.8 TB/s (conversions to f16).
//
// Lanes: with g = lane / 4 and q = lane % 4, a lane holds 16 bytes of weight
// rows g and g + 8 per 64-byte chunk and the same bytes of token row g. Which
// of them feeds which k of the instruction does not matter as long as both
// operands agree, so whole vectors are loaded. MX takes 8 bytes of each
// 32-element block instead, so that an instruction stays within one block.
// NVFP4: e2m1 times its ue4m3 scale is exact in f16 (6 significand bits), so
// both operands become f16 and the block scales need no place in the sum.
#include <cuda_fp16.h>

#include "moe_few.h"
#include "ptx_sm100.cuh"
#include "rowquant.cuh"

namespace mgq {
namespace {

constexpr int kSmallThreads = 256, kWarps = 8;

using ptx::grid_launch;
using ptx::grid_wait;

// Weights are read once: past L1. (Here as everywhere in this file plain loads,
// not those of the read-only path: the first launch may start while the one
// before it still writes what it reads.)
__device__ __forceinline__ uint4 ldw16(const uint8_t* p) {
  uint4 r;
  asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w)
               : "l"(p));
  return r;
}
__device__ __forceinline__ uint2 ldw8(const uint8_t* p) {
  uint2 r;
  asm volatile("ld.global.L1::no_allocate.v2.u32 {%0, %1}, [%2];" : "=r"(r.x), "=r"(r.y) : "l"(p));
  return r;
}
// d += A (16 x 32, e4m3) B (32 x 8, e4m3)
__device__ __forceinline__ void mma_e4m3(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k32.row.col.f32.e4m3.e4m3.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// d += A (16 x 16, f16) B (16 x 8, f16)
__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// byte b of w: two e2m1 values as f16x2 (element 2b in the low half)
__device__ __forceinline__ void e2m1x8_to_f16(uint32_t w, uint32_t (&h)[4]) {
  asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\tmov.b32 {b0, b1, b2, b3}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, b0;\n\tcvt.rn.f16x2.e2m1x2 %1, b1;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, b2;\n\tcvt.rn.f16x2.e2m1x2 %3, b3;\n\t}"
      : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
      : "r"(w));
}
// Two float values as the f16x2 of the e2m1 values nearest to them. (Casts and
// conversions back stay two by two: with four bytes packed into a word between
// them the compiler dropped the second.)
__device__ __forceinline__ uint32_t round_e2m1_f16x2(float lo, float hi) {
  uint32_t r;
  asm("{\n\t.reg .b8 b;\n\tcvt.rn.satfinite.e2m1x2.f32 b, %2, %1;\n\tcvt.rn.f16x2.e2m1x2 %0, b;\n\t}"
      : "=r"(r)
      : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ uint32_t e4m3x2_to_f16(uint32_t two) {
  uint32_t r;
  asm("{\n\t.reg .b16 t;\n\tcvt.u16.u32 t, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, t;\n\t}" : "=r"(r) : "r"(two));
  return r;
}
__device__ __forceinline__ uint32_t hmul2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
// the f16x2 of both halves equal to the low (high) half of s
__device__ __forceinline__ uint32_t dup_lo(uint32_t s) { return __byte_perm(s, s, 0x1010); }
__device__ __forceinline__ uint32_t dup_hi(uint32_t s) { return __byte_perm(s, s, 0x3232); }
// value of the E8M0 code in byte j: its exponent field. (Code 0, 2^-127, reads
// as 0: the codes of such a block stand for less than 2^-118. Code 255, NaN,
// reads as infinity: the element codes beside it are NaN themselves.)
__device__ __forceinline__ float e8m0(uint32_t four, int j) {
  return __uint_as_float((j == 3 ? four >> 1 : four << (23 - 8 * j)) & 0x7F800000u);
}

struct Operand {          // the tokens' operand: x or h, rows in expert order
  const uint8_t* codes;   // FP8 codes [R][K]; NVFP4: f16 values [R][K]
  const void* scales;     // MX: E8M0 [R][K / 32]; 1x128: float32 [R][K / 128]
};
struct Weight {
  const uint8_t* codes;
  int64_t ld;             // bytes per row
  const uint8_t* sf;      // MX, NVFP4: tiled scales
  int64_t sf_kb4;
  const float* s;         // per tensor s, NVFP4 s_g, 1x128: scale_inv [.][K / 128]
};

// ---- routing of at most 64 entries ----------------------------------------------

struct Routing {
  int idx[64], first[64];   // idx: -1 out of range, -2 named before by the same token
};
// The ids, and (PROBS) the probability of each: its own and those of the token's
// later mentions of the expert. Eight lanes take a token's entries, so that
// mentions meet by shuffles.
template <bool PROBS>
__device__ __forceinline__ void load_routing(Routing& r, const int32_t* idx, int T, int k, int E, const float* probs,
                                             float* prob) {
  if (threadIdx.x >= 64) return;
  const int t = threadIdx.x >> 3, j = threadIdx.x & 7, i = t * k + j;
  const bool live = t < T && j < k;
  const int e = live ? idx[i] : -1;
  float p = PROBS && live ? probs[i] : 0.0f;
  const float own = p;
  bool again = false;
#pragma unroll
  for (int d = 1; d < 8; ++d) {
    const int f = __shfl_up_sync(0xFFFFFFFFu, e, d, 8);
    again |= d <= j && f == e;
    if (PROBS) {
      const int g = __shfl_down_sync(0xFFFFFFFFu, e, d, 8);
      const float q = __shfl_down_sync(0xFFFFFFFFu, own, d, 8);
      if (d + j < 8 && g == e) p += q;
    }
  }
  if (live) {
    r.idx[i] = e < 0 || e >= E ? -1 : again ? -2 : e;
    if (PROBS) prob[i] = p;
  }
}
// rows of lower experts, earlier rows of entry i's own, all rows of its own
__device__ __forceinline__ void place(const Routing& r, int R, int i, int& before, int& same, int& n) {
  const int e = r.idx[i];
  before = same = n = 0;
  for (int j = 0; j < R; ++j) {
    const int f = r.idx[j];
    before += f >= 0 && f < e;
    n += f == e;
    same += f == e && j < i;
  }
}

struct SmallArgs {
  const uint16_t* x;
  const int32_t* idx;
  const float* probs;
  int T, k, E, H, F;
  const float* x_scale;
  const float* h_scale;
  uint8_t* hq;
  void* hs;
  Weight w1, w2;
  uint16_t* out;
  int* err;
};

// ---- one unit: 128 bytes of the contraction of 16 weight rows ------------------

// the lane's 32 bytes of a weight row (or of a token row's FP8 codes)
template <int KIND>
__device__ __forceinline__ void load_unit(const uint8_t* row, int q, uint32_t (&w)[8]) {
#pragma unroll
  for (int c = 0; c < 2; ++c) {
    if (KIND == kMX) {
      const uint2 a = ldw8(row + c * 64 + 8 * q), b = ldw8(row + c * 64 + 32 + 8 * q);
      w[4 * c] = a.x, w[4 * c + 1] = a.y, w[4 * c + 2] = b.x, w[4 * c + 3] = b.y;
    } else {
      const uint4 a = ldw16(row + c * 64 + 16 * q);
      w[4 * c] = a.x, w[4 * c + 1] = a.y, w[4 * c + 2] = a.z, w[4 * c + 3] = a.w;
    }
  }
}
// block scales of the lane's row for unit u: MX four E8M0 bytes; NVFP4 the two
// ue4m3 of each chunk that its 16 bytes lie in
template <int KIND>
__device__ __forceinline__ void load_sf(const Weight& w, int64_t row, int u, int q, uint32_t (&s)[2]) {
  const uint8_t* t = w.sf + (row >> 7) * w.sf_kb4 * 512 + (row & 31) * 16 + ((row >> 5) & 3) * 4;
  if (KIND == kMX) {
    s[0] = *reinterpret_cast<const uint32_t*>(t + static_cast<int64_t>(u) * 512);
  } else {
#pragma unroll
    for (int c = 0; c < 2; ++c)
      s[c] = *reinterpret_cast<const uint32_t*>(t + (static_cast<int64_t>(u) * 4 + 2 * c + (q >> 1)) * 512) >>
             (16 * (q & 1)) & 0xFFFFu;
  }
}

// The tokens' side of a unit, shared by the tiles of the warp.
template <int KIND>
struct Tokens {
  uint32_t b[KIND == kNV ? 32 : 8];
  float s[KIND == kMX ? 8 : KIND == kBLK ? 2 : 1];     // MX: 4 blocks x 2 tokens; 1x128: 2 tokens

  __device__ __forceinline__ void load(const Operand& o, int64_t row0, int n, int K, int u, int g, int q) {
    // (h is written by the launch before: plain loads)
    if (KIND == kNV) {
#pragma unroll
      for (int c = 0; c < 2; ++c)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          uint4 v = make_uint4(0, 0, 0, 0);
          if (g < n)
            v = *(reinterpret_cast<const uint4*>(o.codes + ((row0 + g) * K + u * 256 + c * 128 + q * 32) * 2) + j);
          b[16 * c + 4 * j] = v.x, b[16 * c + 4 * j + 1] = v.y, b[16 * c + 4 * j + 2] = v.z, b[16 * c + 4 * j + 3] = v.w;
        }
      return;
    }
    const uint8_t* row = o.codes + (row0 + g) * K + u * 128;
#pragma unroll
    for (int j = 0; j < 8; ++j) b[j] = 0u;
    if (g < n) {
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        if (KIND == kMX) {
          const uint2 x = *reinterpret_cast<const uint2*>(row + c * 64 + 8 * q);
          const uint2 y = *reinterpret_cast<const uint2*>(row + c * 64 + 32 + 8 * q);
          b[4 * c] = x.x, b[4 * c + 1] = x.y, b[4 * c + 2] = y.x, b[4 * c + 3] = y.y;
        } else {
          const uint4 x = *reinterpret_cast<const uint4*>(row + c * 64 + 16 * q);
          b[4 * c] = x.x, b[4 * c + 1] = x.y, b[4 * c + 2] = x.z, b[4 * c + 3] = x.w;
        }
      }
    }
    if (KIND == kMX || KIND == kBLK) {
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        const int tok = 2 * q + t;
        const int64_t at = (row0 + tok) * (K / 128) + u;
        if (KIND == kMX) {
          const uint32_t e = tok < n ? static_cast<const uint32_t*>(o.scales)[at] : 0u;
#pragma unroll
          for (int j = 0; j < 4; ++j) s[(2 * j + t) % (KIND == kMX ? 8 : 1)] = e8m0(e, j);
        } else {
          s[t % (KIND == kBLK ? 2 : 1)] = tok < n ? static_cast<const float*>(o.scales)[at] : 0.0f;
        }
      }
    }
  }
};

// One unit of up to eight tokens' x, quantised by the warp into its own piece of
// shared memory: all lanes share each token's elements (8 a lane for NVFP4, 4
// else), whichever of them the tokens' operand will need.
template <int KIND>
struct XUnit {
  static constexpr int kEl = KIND == kNV ? 8 : 4;
  // bytes of a token: the operand, 16 to spread the rows over the banks
  static constexpr int kRow = (KIND == kNV ? 512 : 128) + 16;
  uint4 raw[8];                            // (two words used by the FP8 kinds)

  // `x` of the expert's n tokens (rows s_tok of a.x)
  __device__ __forceinline__ void load(const uint16_t* x, const int* tok, int n, int H, int u, int lane) {
#pragma unroll
    for (int t = 0; t < 8; ++t) {
      if (t >= n) break;
      const uint16_t* p = x + static_cast<int64_t>(tok[t]) * H + u * 32 * kEl + lane * kEl;
      if (KIND == kNV) {
        raw[t] = *reinterpret_cast<const uint4*>(p);
      } else {
        const uint2 v = *reinterpret_cast<const uint2*>(p);
        raw[t].x = v.x, raw[t].y = v.y;
      }
    }
  }
  // the recipe's rule; then the tokens' operand of this lane
  __device__ __forceinline__ void quantize(uint8_t* sm, float* sc_sm, int n, float scale, int lane, Tokens<KIND>& o) const {
    const int g = lane >> 2, q = lane & 3;
    __syncwarp();                          // the last unit's reads are done
#pragma unroll
    for (int t = 0; t < 8; ++t) {
      if (t >= n) break;
      float f[kEl];
      f[0] = bf16_lo(raw[t].x), f[1] = bf16_hi(raw[t].x), f[2] = bf16_lo(raw[t].y), f[3] = bf16_hi(raw[t].y);
      if constexpr (KIND == kNV)
        f[4] = bf16_lo(raw[t].z), f[5] = bf16_hi(raw[t].z), f[6] = bf16_lo(raw[t].w), f[7] = bf16_hi(raw[t].w);
      uint32_t m = absmax_bits_f32(f, kEl);
      if constexpr (KIND == kNV) {
        m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, 1));
        const float sc = ue4m3_value(cvt_ue4m3(__fmul_rn(__fdiv_rn(__uint_as_float(m), 6.0f), scale)));
        const float r = sc == 0.0f ? 0.0f : __fdiv_rn(scale, sc);
        const uint32_t s2 = dup_lo(static_cast<uint32_t>(__half_as_ushort(__float2half_rn(sc))));
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
          w[i] = hmul2(round_e2m1_f16x2(__fmul_rn(f[2 * i], r), __fmul_rn(f[2 * i + 1], r)), s2);
        *reinterpret_cast<uint4*>(sm + t * kRow + lane * 16) = make_uint4(w[0], w[1], w[2], w[3]);
      } else {
        float mult = scale;
        if constexpr (KIND == kMX) {
          m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, 1));
          m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, 2));
          m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, 4));
          const int e = mx_exponent(m, 8, true);
          mult = mx_multiplier(e);
          if ((lane & 7) == 0) sc_sm[t * 4 + (lane >> 3)] = e8m0(mx_scale_code(e), 0);
        }
        if constexpr (KIND == kBLK) {
          mult = blk_scale_few(__reduce_max_sync(0xFFFFFFFFu, m));
          if (lane == 0) sc_sm[t] = __fdiv_rn(1.0f, mult);
        }
        *reinterpret_cast<uint32_t*>(sm + t * kRow + lane * 4) = cvt_fp8x4_mul<MGQ_E4M3>(f[0], f[1], f[2], f[3], mult);
      }
    }
    __syncwarp();
    const uint8_t* row = sm + g * kRow;
    constexpr int kWords = KIND == kNV ? 32 : 8;
#pragma unroll
    for (int j = 0; j < kWords; ++j) o.b[j] = 0u;
    if (g < n) {
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        if constexpr (KIND == kNV) {
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const uint4 v = *reinterpret_cast<const uint4*>(row + c * 256 + q * 64 + j * 16);
            o.b[16 * c + 4 * j] = v.x, o.b[16 * c + 4 * j + 1] = v.y, o.b[16 * c + 4 * j + 2] = v.z,
                              o.b[16 * c + 4 * j + 3] = v.w;
          }
        } else if constexpr (KIND == kMX) {
          const uint2 x = *reinterpret_cast<const uint2*>(row + c * 64 + 8 * q);
          const uint2 y = *reinterpret_cast<const uint2*>(row + c * 64 + 32 + 8 * q);
          o.b[4 * c] = x.x, o.b[4 * c + 1] = x.y, o.b[4 * c + 2] = y.x, o.b[4 * c + 3] = y.y;
        } else {
          const uint4 x = *reinterpret_cast<const uint4*>(row + c * 64 + 16 * q);
          o.b[4 * c] = x.x, o.b[4 * c + 1] = x.y, o.b[4 * c + 2] = x.z, o.b[4 * c + 3] = x.w;
        }
      }
    }
    if constexpr (KIND == kMX || KIND == kBLK) {
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        const bool on = 2 * q + t < n;
        if constexpr (KIND == kMX) {
#pragma unroll
          for (int j = 0; j < 4; ++j) o.s[2 * j + t] = on ? sc_sm[(2 * q + t) * 4 + j] : 0.0f;
        } else {
          o.s[t] = on ? sc_sm[2 * q + t] : 0.0f;
        }
      }
    }
  }
};

// acc += the unit's product of 16 weight rows (words w0: row g, w1: row g + 8)
// and the tokens. sw: 1x128 weight scale.
template <int KIND>
__device__ __forceinline__ void unit_mma(float (&acc)[4], const uint32_t (&w0)[8], const uint32_t (&w1)[8],
                                         const uint32_t (&f0)[2], const uint32_t (&f1)[2], const Tokens<KIND>& t,
                                         float sw) {
  if (KIND == kNV) {
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      const uint32_t s0 = e4m3x2_to_f16(f0[c]), s1 = e4m3x2_to_f16(f1[c]);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        uint32_t h0[4], h1[4];
        e2m1x8_to_f16(w0[4 * c + j], h0);
        e2m1x8_to_f16(w1[4 * c + j], h1);
        const uint32_t m0 = j < 2 ? dup_lo(s0) : dup_hi(s0), m1 = j < 2 ? dup_lo(s1) : dup_hi(s1);
#pragma unroll
        for (int i = 0; i < 4; i += 2)
          mma_f16(acc, hmul2(h0[i], m0), hmul2(h1[i], m1), hmul2(h0[i + 1], m0), hmul2(h1[i + 1], m1),
                  t.b[(16 * c + 4 * j + i) % (KIND == kNV ? 32 : 8)], t.b[(16 * c + 4 * j + i + 1) % (KIND == kNV ? 32 : 8)]);
      }
    }
  } else if (KIND == kMX) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      float d[4] = {0.0f, 0.0f, 0.0f, 0.0f};
      mma_e4m3(d, w0[2 * j], w1[2 * j], w0[2 * j + 1], w1[2 * j + 1], t.b[2 * j], t.b[2 * j + 1]);
      const float a = e8m0(f0[0], j), b = e8m0(f1[0], j);
      const float x = t.s[(2 * j) % (KIND == kMX ? 8 : 1)], y = t.s[(2 * j + 1) % (KIND == kMX ? 8 : 1)];
      acc[0] = fmaf(d[0], a * x, acc[0]);
      acc[1] = fmaf(d[1], a * y, acc[1]);
      acc[2] = fmaf(d[2], b * x, acc[2]);
      acc[3] = fmaf(d[3], b * y, acc[3]);
    }
  } else {
    float d[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    float (&to)[4] = KIND == kTEN ? acc : d;
#pragma unroll
    for (int j = 0; j < 4; ++j)
      mma_e4m3(to, w0[2 * j], w1[2 * j], w0[2 * j + 1], w1[2 * j + 1], t.b[2 * j], t.b[2 * j + 1]);
    if (KIND == kBLK) {
      const float x = sw * t.s[0], y = sw * t.s[1 % (KIND == kBLK ? 2 : 1)];
      acc[0] = fmaf(d[0], x, acc[0]);
      acc[1] = fmaf(d[1], y, acc[1]);
      acc[2] = fmaf(d[2], x, acc[2]);
      acc[3] = fmaf(d[3], y, acc[3]);
    }
  }
}

// ---- gate, up, SwiGLU -----------------------------------------------------------

// ffn rows of a CTA of the gate/up kernel: an MX block, a quarter of a 1x128
// block, one NVFP4 block
__host__ __device__ constexpr int ffn_rows(int kind) { return kind == kNV ? 16 : 32; }

// GW: warps of a CTA
template <int KIND, int GW>
__global__ void __launch_bounds__(32 * GW, 16 / GW) small_gateup_kernel(SmallArgs a) {
  constexpr int FR = ffn_rows(KIND), TS = FR / 16;     // 16-row tiles of each side
  __shared__ Routing rt;
  __shared__ int sel[3], s_tok[8];
  __shared__ float red[GW][8][2 * FR + 1];
  __shared__ __align__(16) uint8_t xsm[GW][8 * XUnit<KIND>::kRow];
  __shared__ float xsc[GW][KIND == kMX ? 32 : 8];
  __shared__ uint32_t cmax[8];
  grid_wait();
  grid_launch();
  const int R = a.T * a.k, warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, q = lane & 3;
  load_routing<false>(rt, a.idx, a.T, a.k, a.E, nullptr, nullptr);
  if (threadIdx.x == 0) sel[0] = -1, sel[2] = 0;
  __syncthreads();
  int before = 0, same = 0, n = 0;
  const bool in = static_cast<int>(threadIdx.x) < R;
  const bool mine = in && rt.idx[threadIdx.x] >= 0;
  if (in && rt.idx[threadIdx.x] == -1 && blockIdx.x == 0 && blockIdx.y == 0) report(a.err, MGQ_ERR_DEVICE_INDEX);
  if (mine) place(rt, R, threadIdx.x, before, same, n);
  if (threadIdx.x < 64) rt.first[threadIdx.x] = mine && same == 0;
  __syncthreads();
  if (mine && same == 0) {
    int rank = 0;
    for (int j = 0; j < R; ++j) rank += rt.first[j] && rt.idx[j] < rt.idx[threadIdx.x];
    if (rank == static_cast<int>(blockIdx.y)) sel[0] = rt.idx[threadIdx.x], sel[1] = before, sel[2] = n;
  }
  __syncthreads();
  n = min(sel[2], 8);                      // (at most T; the bound spares registers)
  if (n == 0) return;                      // fewer experts picked than the grid allows for
  const int e = sel[0], row0 = sel[1];
  if (mine && rt.idx[threadIdx.x] == e) s_tok[same] = threadIdx.x / a.k;
  __syncthreads();
  const int64_t f0 = static_cast<int64_t>(blockIdx.x) * FR, wrow = static_cast<int64_t>(e) * 2 * a.F + f0;
  const int units = a.H / (KIND == kNV ? 256 : 128);
  const int u0 = warp * units / GW, u1 = (warp + 1) * units / GW;
  // (all scales up front: behind the reduction's barrier their loads would be waited for)
  const bool scaled = KIND == kTEN || KIND == kNV;
  const float sx = scaled ? *a.x_scale : 1.0f, sh = scaled ? *a.h_scale : 1.0f, s_w = scaled ? a.w1.s[e] : 1.0f;
  float acc[2 * TS][4];
#pragma unroll
  for (int i = 0; i < 2 * TS; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) acc[i][j] = 0.0f;
  for (int u = u0; u < u1; ++u) {
    uint32_t w[2 * TS][2][8], sf[2 * TS][2][2];
    float sw[2] = {1.0f, 1.0f};
#pragma unroll
    for (int i = 0; i < 2 * TS; ++i)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int64_t row = wrow + (i / TS) * a.F + (i % TS) * 16 + h * 8 + g;
        load_unit<KIND>(a.w1.codes + row * a.w1.ld + u * 128, q, w[i][h]);
        if (KIND == kMX || KIND == kNV) load_sf<KIND>(a.w1, row, u, q, sf[i][h]);
      }
    if (KIND == kBLK) {
      sw[0] = a.w1.s[(wrow >> 7) * (a.H / 128) + u];
      sw[1] = a.w1.s[((wrow + a.F) >> 7) * (a.H / 128) + u];
    }
    XUnit<KIND> xu;
    xu.load(a.x, s_tok, n, a.H, u, lane);
    Tokens<KIND> t;
    xu.quantize(xsm[warp], xsc[warp], n, sx, lane, t);
#pragma unroll
    for (int i = 0; i < 2 * TS; ++i) unit_mma<KIND>(acc[i], w[i][0], w[i][1], sf[i][0], sf[i][1], t, sw[i / TS]);
  }
#pragma unroll
  for (int i = 0; i < 2 * TS; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) red[warp][2 * q + (j & 1)][16 * i + 8 * (j >> 1) + g] = acc[i][j];
  __syncthreads();
  // thread: one ffn row of one token
  const int tok = threadIdx.x / FR, f = threadIdx.x % FR;
  const bool on = tok < n;
  const int64_t r = row0 + tok;
  float h = 0.0f;
  if (on) {
    float gt = 0.0f, up = 0.0f;
#pragma unroll
    for (int w = 0; w < GW; ++w) {
      gt += red[w][tok][f];
      up += red[w][tok][FR + f];
    }
    float alpha = 1.0f;
    if (scaled) alpha = 1.0f / (sx * s_w);
    h = swiglu_f32(gt * alpha, up * alpha);
  }
  uint32_t m = __float_as_uint(h) & 0x7FFFFFFFu;
  if (KIND == kBLK) {
    // the block's other three quarters are the cluster's other CTAs
    m = __reduce_max_sync(0xFFFFFFFFu, m);
    if (f == 0) cmax[tok] = m;
    ptx::cluster_sync();
    const uint32_t at = ptx::smem_u32(&cmax[tok]);
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      uint32_t o;
      asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(o) : "r"(ptx::mapa_shared(at, c)) : "memory");
      m = max(m, o);
    }
    ptx::cluster_sync();                   // nobody leaves while its maximum may still be read
  }
  if (KIND == kNV) {
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
    const float sc = ue4m3_value(cvt_ue4m3(__fmul_rn(__fdiv_rn(__uint_as_float(m), 6.0f), sh)));
    const float v = __fmul_rn(h, sc == 0.0f ? 0.0f : __fdiv_rn(sh, sc));
    const uint32_t two = round_e2m1_f16x2(v, 0.0f);
    const __half hv = __hmul(__ushort_as_half(static_cast<uint16_t>(two)), __float2half_rn(sc));
    if (on) reinterpret_cast<__half*>(a.hq)[r * a.F + f0 + f] = hv;
  } else if (on) {                         // (a warp is one token)
    float mult;
    if (KIND == kMX) {
      const int ex = mx_exponent(__reduce_max_sync(0xFFFFFFFFu, m), 8, true);
      mult = mx_multiplier(ex);
      if (f == 0) static_cast<uint8_t*>(a.hs)[r * (a.F / 32) + blockIdx.x] = static_cast<uint8_t>(mx_scale_code(ex));
    } else if (KIND == kBLK) {
      mult = blk_scale_few(m);
      if (f == 0 && (blockIdx.x & 3) == 0)
        static_cast<float*>(a.hs)[r * (a.F / 128) + (blockIdx.x >> 2)] = __fdiv_rn(1.0f, mult);
    } else {
      mult = sh;
    }
    a.hq[r * a.F + f0 + f] = static_cast<uint8_t>(cvt_e4m3x2(__fmul_rn(h, mult), 0.0f));
  }
}

// ---- down, probabilities, sum over the experts ----------------------------------

template <int KIND>
__global__ void __launch_bounds__(kSmallThreads, 2) small_down_kernel(SmallArgs a) {
  constexpr int UN = 4;                    // units in flight
  __shared__ Routing rt;
  __shared__ int l_e[64], l_row[64], l_n[64], s_tok[64];
  __shared__ float s_p[64], prob[64];
  __shared__ int s_na;
  __shared__ float part[kWarps][8][17];
  grid_launch();
  const int R = a.T * a.k, warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, q = lane & 3;
  load_routing<true>(rt, a.idx, a.T, a.k, a.E, a.probs, prob);
  for (int i = threadIdx.x; i < kWarps * 8 * 17; i += kSmallThreads) (&part[0][0][0])[i] = 0.0f;
  if (threadIdx.x == 0) s_na = 0;
  __syncthreads();
  int before = 0, same = 0, n = 0;
  const bool mine = static_cast<int>(threadIdx.x) < R && rt.idx[threadIdx.x] >= 0;
  if (mine) {
    place(rt, R, threadIdx.x, before, same, n);
    s_tok[before + same] = threadIdx.x / a.k;
    s_p[before + same] = prob[threadIdx.x];
  }
  if (threadIdx.x < 64) rt.first[threadIdx.x] = mine && same == 0;
  __syncthreads();
  if (mine && same == 0) {
    int rank = 0;
    for (int j = 0; j < R; ++j) rank += rt.first[j] && rt.idx[j] < rt.idx[threadIdx.x];
    l_e[rank] = rt.idx[threadIdx.x];
    l_row[rank] = before;
    l_n[rank] = n;
    atomicAdd(&s_na, 1);
  }
  __syncthreads();
  const int64_t h0 = static_cast<int64_t>(blockIdx.x) * 16;
  const int units = a.F / (KIND == kNV ? 256 : 128), all = s_na * units;
  int u = warp * all / kWarps;
  const int u1 = (warp + 1) * all / kWarps;
  int at = u / units;
  const Operand x{a.hq, a.hs};
  bool waited = false;
  while (u < u1) {
    const int e = l_e[at], row0 = l_row[at], n = min(l_n[at], 8);
    const int64_t wrow = static_cast<int64_t>(e) * a.H + h0 + g;
    const int end = min(u1, (at + 1) * units) - at * units;
    int k0 = u - at * units;
    u += end - k0;
    float acc[4] = {0.0f, 0.0f, 0.0f, 0.0f}, alpha = 1.0f;
    if (KIND == kTEN || KIND == kNV) alpha = 1.0f / (*a.h_scale * a.w2.s[e]);
    for (; k0 < end; k0 += UN) {
      uint32_t w[UN][2][8], sf[UN][2][2];
      float sw[UN];
#pragma unroll
      for (int i = 0; i < UN; ++i) {
        if (k0 + i >= end) break;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          load_unit<KIND>(a.w2.codes + (wrow + 8 * h) * a.w2.ld + (k0 + i) * 128, q, w[i][h]);
          if (KIND == kMX || KIND == kNV) load_sf<KIND>(a.w2, wrow + 8 * h, k0 + i, q, sf[i][h]);
        }
        sw[i] = KIND == kBLK ? a.w2.s[((static_cast<int64_t>(e) * a.H + h0) >> 7) * (a.F / 128) + k0 + i] : 1.0f;
      }
      if (!waited) {
        grid_wait();
        waited = true;
      }
#pragma unroll
      for (int i = 0; i < UN; ++i) {
        if (k0 + i >= end) break;
        Tokens<KIND> t;
        t.load(x, row0, n, a.F, k0 + i, g, q);
        unit_mma<KIND>(acc, w[i][0], w[i][1], sf[i][0], sf[i][1], t, sw[i]);
      }
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int c = 2 * q + (j & 1);
      if (c < n) part[warp][s_tok[row0 + c]][g + 8 * (j >> 1)] += acc[j] * alpha * s_p[row0 + c];
    }
    __syncwarp();
    ++at;
  }
  if (!waited) grid_wait();
  __syncthreads();
  const int t = threadIdx.x >> 4, r = threadIdx.x & 15;
  if (t < a.T) {
    float o = 0.0f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) o += part[w][t][r];
    a.out[static_cast<int64_t>(t) * a.H + h0 + r] = __bfloat16_as_ushort(__float2bfloat16_rn(o));
  }
}

// ---- host side --------------------------------------------------------------------

template <int KIND>
int run_small(const SmallArgs& a, cudaStream_t s) {
  const int R = a.T * a.k;
  const dim3 grid(a.F / ffn_rows(KIND), R < a.E ? R : a.E);
  // NVFP4's CTAs of 16 rows: with four warps each, twice as many are on the GPU
  // at once. Taken where eight warps need a second wave (384 CTAs: 13.7 / 12.2 us
  // at H 2048; 128 CTAs at H 4096: 10.1 / 13.9).
  auto gateup = small_gateup_kernel<KIND, 8>;
  int warps = 8;
  if constexpr (KIND == kNV) {
    if (static_cast<int64_t>(grid.x) * grid.y > 2 * num_sms()) gateup = small_gateup_kernel<KIND, 4>, warps = 4;
  }
  if (!launch_after(gateup, grid, 32 * warps, 0, KIND == kBLK ? 4 : 1, s, a)) return MGQ_ERR_CUDA;
  if (!launch_after(small_down_kernel<KIND>, dim3(a.H / 16), kSmallThreads, 0, 1, s, a)) return MGQ_ERR_CUDA;
  return MGQ_OK;
}

Weight weight_of(const mgq_operand* W, int kind) {
  Weight w{};
  w.codes = static_cast<const uint8_t*>(W->data);
  w.ld = kind == kNV ? W->ld / 2 : W->ld;
  w.sf = static_cast<const uint8_t*>(W->scale);
  w.sf_kb4 = W->ld / (kind == kNV ? 64 : 128);
  w.s = kind == kNV ? W->global_scale : static_cast<const float*>(W->scale);
  return w;
}

struct SmallLayout {
  int64_t hq, hs, total;
};
SmallLayout small_layout(int R, int64_t F, int kind) {
  SmallLayout l{};
  int64_t at = 0;
  auto take = [&](int64_t bytes) {
    const int64_t o = at;
    at += (bytes + 255) / 256 * 256;
    return o;
  };
  const int per = kind == kNV ? 2 : 1;
  l.hq = take(R * F * per);
  l.hs = take(R * (F / 128) * 4);
  l.total = at;
  return l;
}

}  // namespace

size_t few_small_workspace(int T, int k, int64_t F, int kind) {
  return static_cast<size_t>(small_layout(T * k, F, kind).total);
}

int few_small_forward(int kind, const void* x, int T, int64_t H, int64_t F, const int32_t* idx, const float* probs, int k,
                      int E, const mgq_operand* W1, const mgq_operand* W2, const float* x_scale, const float* h_scale,
                      void* out, uint8_t* ws, cudaStream_t s) {
  const SmallLayout l = small_layout(T * k, F, kind);
  SmallArgs a{};
  a.x = static_cast<const uint16_t*>(x);
  a.idx = idx;
  a.probs = probs;
  a.T = T;
  a.k = k;
  a.E = E;
  a.H = static_cast<int>(H);
  a.F = static_cast<int>(F);
  a.x_scale = x_scale;
  a.h_scale = h_scale;
  a.hq = ws + l.hq;
  a.hs = ws + l.hs;
  a.w1 = weight_of(W1, kind);
  a.w2 = weight_of(W2, kind);
  a.out = static_cast<uint16_t*>(out);
  a.err = error_word();
  switch (kind) {
    case kMX: return run_small<kMX>(a, s);
    case kNV: return run_small<kNV>(a, s);
    case kBLK: return run_small<kBLK>(a, s);
    default: return run_small<kTEN>(a, s);
  }
}

}  // namespace mgq
