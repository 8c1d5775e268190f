// int8 codes to f16 operands of the tensor cores: a byte b becomes f16 by one
// permutation and one subtraction for two, 0x6400 | (b ^ 0x80) being 1152 + b.
#pragma once
#include <cuda_fp16.h>

#include "ptx_sm100.cuh"

namespace mgq {
namespace {

constexpr int kBK8 = 128;                          // elements (bytes) of the contraction a stage

// 16 codes -> 16 f16 values in 8 words
__device__ __forceinline__ void widen16(const uint4& c, uint32_t* o) {
  const uint32_t w[4] = {c.x, c.y, c.z, c.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t u = w[i] ^ 0x80808080u;
    uint32_t lo = __byte_perm(u, 0x64646464u, 0x4140), hi = __byte_perm(u, 0x64646464u, 0x4342);
    const __half2 base = __halves2half2(__ushort_as_half(0x6480), __ushort_as_half(0x6480));   // 1152
    __half2 a = __hsub2(*reinterpret_cast<__half2*>(&lo), base), b = __hsub2(*reinterpret_cast<__half2*>(&hi), base);
    o[2 * i] = *reinterpret_cast<uint32_t*>(&a);
    o[2 * i + 1] = *reinterpret_cast<uint32_t*>(&b);
  }
}

// One row's 64 codes of half h of a stage: 4 of the row's 8 chunks of 16 bytes, in
// the 128-byte swizzle that the TMA wrote.
__device__ __forceinline__ void load_codes(const uint8_t* tile, uint32_t row, int h, uint4 (&c)[4]) {
#pragma unroll
  for (int j = 0; j < 4; ++j) c[j] = *reinterpret_cast<const uint4*>(tile + row * 128 + (((4 * h + j) ^ (row & 7)) << 4));
}
// ... as the MMA's A operand in tensor memory: lane = row, 32 columns of two elements
__device__ __forceinline__ void codes_to_tmem(const uint4 (&c)[4], uint32_t taddr) {
  uint32_t o[32];
#pragma unroll
  for (int j = 0; j < 4; ++j) widen16(c[j], o + 8 * j);
  ptx::tmem_st_32x32b_x32(taddr, o);
}
// the same in two pieces, for warps with few registers
__device__ __forceinline__ void codes_to_tmem_halves(const uint4 (&c)[4], uint32_t taddr) {
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    uint32_t o[16];
    widen16(c[2 * h], o);
    widen16(c[2 * h + 1], o + 8);
    ptx::tmem_st_32x32b_x16(taddr + 16 * h, o);
  }
}
// ... as a K-major operand in shared memory: rows of 64 elements, 128-byte swizzle
__device__ __forceinline__ void codes_to_smem(const uint4 (&c)[4], uint8_t* tile, uint32_t row) {
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    uint32_t o[8];
    widen16(c[j], o);
    uint8_t* dst = tile + row * 128;
    *reinterpret_cast<uint4*>(dst + (((2 * j) ^ (row & 7)) << 4)) = make_uint4(o[0], o[1], o[2], o[3]);
    *reinterpret_cast<uint4*>(dst + (((2 * j + 1) ^ (row & 7)) << 4)) = make_uint4(o[4], o[5], o[6], o[7]);
  }
}

}  // namespace
}  // namespace mgq
