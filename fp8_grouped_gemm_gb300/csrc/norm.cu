// Residual addition + RMSNorm with an 8-bit output, and its gradient.
//
// Forward, per row:  s = x + r,  rstd = 1 / sqrt(mean(s^2) + eps),
//                    y = s rstd w,  codes = Q(y) from the float32 y.
// Backward, per row: xh = s rstd,  g = dy w,
//                    dx = rstd (g - xh mean(g xh)) + dsum,
//                    dw = sum over rows of dy xh.
//
// Both are bound by memory: every element is read once, held in registers
// between the row's reduction and its output, and written once. A CTA owns
// whole rows (a thread takes 16-byte chunks tid, tid + threads, ... so that
// each warp access covers 512 contiguous bytes); four adjacent lanes hold one
// 32-element MX block and sixteen one 1x128 block, so a block's amax is two or
// four shuffles.
//
// A row's loads cannot overlap its own reduction, so with many rows a CTA
// streams them: bulk copies bring the next rows into a ring of shared-memory
// slots while the current one is reduced and written.
//
// Measured, with residual, sum, y and MXFP8 codes: a row of 4096 in 2.6 us, all
// of it the launch, one trip to memory and the reduction; 1003 x 5120 (1x128,
// no residual) in 6.6 us, 3.9 TB/s; 16384 x 4096 in 101 us, 6.0 TB/s of the
// 6.8 that a plain copy reaches (two streams read, three written). Backward with
// dsum, 16384 x 4096: 80 us, 6.7 TB/s; 333 x 2048 in 5.0 us, two launches in a row.
#include "mgq_internal.h"
#include "ptx_sm100.cuh"
#include "rowquant.cuh"

namespace mgq {
namespace {

constexpr int kNoQuant = -1;

// float32 values of a 16-byte chunk of bf16
__device__ __forceinline__ void unpack8(uint4 w, float* v) {
  v[0] = bf16_lo(w.x); v[1] = bf16_hi(w.x);
  v[2] = bf16_lo(w.y); v[3] = bf16_hi(w.y);
  v[4] = bf16_lo(w.z); v[5] = bf16_hi(w.z);
  v[6] = bf16_lo(w.w); v[7] = bf16_hi(w.w);
}
__device__ __forceinline__ uint4 pack8(const float* v) {
  return make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]),
                    pack_bf16x2(v[6], v[7]));
}

// (These kernels are launched while the one before them may still run. What that
// one can have written is read with plain loads: those of the read-only path ask
// for data that nobody writes while the kernel lives, and nothing but the
// compiler's order would keep them behind the wait.)

// the weight chunk c (8 values) as float32; wf32 selects float32 storage
__device__ __forceinline__ void load_w8(const void* w, bool wf32, int c, float* v) {
  if (wf32) {
    const float4* p = reinterpret_cast<const float4*>(w) + 2 * c;
    const float4 a = p[0], b = p[1];
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
    v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
  } else {
    unpack8(reinterpret_cast<const uint4*>(w)[c], v);
  }
}

// max |v| with NaN winning, as float bits
template <int N>
__device__ __forceinline__ uint32_t absmax(const float* v) {
  float m = 0.0f;
#pragma unroll
  for (int j = 0; j < N; ++j) asm("max.NaN.f32 %0, %0, %1;" : "+f"(m) : "f"(fabsf(v[j])));
  return __float_as_uint(m);
}

// mx_exponent, mx_scale_code and mx_multiplier of an amax in one: a subnormal
// amax lies below the smallest exponent whatever its bits, and a finite one
// never reaches the largest.
__device__ __forceinline__ void mx_scale(uint32_t amax_bits, int emax, int rceil, uint32_t& code, float& mult) {
  const int up = (rceil && (amax_bits & 0x7FFFFFu) > 0x600000u) ? 1 : 0;
  const int c = max(0, static_cast<int>(amax_bits >> 23) - emax + up);      // exponent + 127
  const bool fine = amax_bits < 0x7F800000u;
  code = fine ? static_cast<uint32_t>(c) : 255u;
  mult = __uint_as_float(fine ? static_cast<uint32_t>(254 - c) << 23 : 0x7FC00000u);
}

// Sum over the CTA; `slot` alternates between two shared arrays from one call
// to the next, so that one barrier a call is enough. ANY: `any` becomes true in
// every thread if it is in one.
template <bool ANY>
__device__ __forceinline__ float block_sum(float v, float (*red)[32], int slot, bool& any) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
  const int warp = threadIdx.x >> 5, nw = blockDim.x >> 5;
  if (nw == 1) {
    if (ANY) any = __any_sync(0xFFFFFFFFu, any);
    __syncwarp();
    return v;
  }
  if ((threadIdx.x & 31) == 0) red[slot][warp] = v;
  if (ANY) any = __syncthreads_or(any);
  else __syncthreads();
  float t = (threadIdx.x & 31) < nw ? red[slot][threadIdx.x & 31] : 0.0f;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) t += __shfl_xor_sync(0xFFFFFFFFu, t, o);
  return t;
}

constexpr int kMaxSlots = 8;

struct RingArgs {
  int slots;
  int stall;               // failure-detection test: no row is requested
  uint64_t wait_ns;        // limit of a wait for a row's copies
  int* err;
};

// A ring of row slots filled by bulk copies: NS source rows side by side per
// slot. Thread 0 requests; the barrier that every reduction passes frees a slot.
// A wait that runs out in some threads must not leave the others at a barrier
// or a shuffle: all of them still take part in the row's reduction, whose barrier
// tells every thread whether one gave up.
template <int NS>
struct RowRing {
  uint64_t* full;
  uint8_t* mem;
  uint32_t row_bytes;
  int slots, st, ask;      // slot to read next, slot to fill next
  uint32_t ph;
  int64_t next;            // row to request next

  __device__ __forceinline__ void init(uint8_t* base, uint64_t* bars, const RingArgs& a, uint32_t bytes) {
    full = bars;
    mem = base;
    row_bytes = bytes;
    slots = a.slots;
    st = ask = 0;
    ph = 0;
    next = a.stall ? INT64_MAX : blockIdx.x;
    if (threadIdx.x == 0) {
      for (int i = 0; i < slots; ++i) ptx::mbar_init(&full[i], 1);
      ptx::fence_mbar_init();
    }
    __syncthreads();
  }
  // thread 0: request the next row of each source (null: none)
  __device__ __forceinline__ void request(const uint16_t* const (&src)[NS], int64_t T) {
    if (next >= T) return;
    uint32_t n = 0;
#pragma unroll
    for (int i = 0; i < NS; ++i) n += src[i] ? row_bytes : 0u;
    ptx::mbar_arrive_expect_tx(&full[ask], n);
#pragma unroll
    for (int i = 0; i < NS; ++i)
      if (src[i])
        ptx::bulk_load(mem + (static_cast<size_t>(ask) * NS + i) * row_bytes,
                       reinterpret_cast<const uint8_t*>(src[i]) + next * row_bytes, row_bytes, &full[ask]);
    next += gridDim.x;
    if (++ask == slots) ask = 0;
  }
  __device__ __forceinline__ bool wait(uint64_t limit_ns) { return ptx::mbar_wait(&full[st], ph, limit_ns); }
  __device__ __forceinline__ const uint4* row(int i) const {
    return reinterpret_cast<const uint4*>(mem + (static_cast<size_t>(st) * NS + i) * row_bytes);
  }
  // after a wait that ran out: give the copies in flight a last, short chance
  __device__ __forceinline__ void drain(uint64_t limit_ns) {
    for (int i = 0; i < slots && threadIdx.x == 0; ++i)
      ptx::mbar_wait(&full[(st + i) % slots], ph ^ (st + i >= slots ? 1u : 0u), limit_ns / 100);
  }
  __device__ __forceinline__ void advance() {
    if (++st == slots) st = 0, ph ^= 1;
  }
};

struct NormArgs {
  const uint16_t* x;
  const uint16_t* res;   // or null
  const void* w;
  int wf32;
  int64_t T;
  int H;
  float eps;
  uint16_t* sum;         // or null
  uint16_t* y;           // or null
  uint8_t* codes;
  uint8_t* scales;
  const float* ts;       // per-tensor scale
  float* amax;           // per-tensor amax, or null
  int rceil;
  float* rstd;           // or null
  RingArgs ring;         // streamed
  int wide;              // streamed: 32-byte aligned bf16 outputs
};

// rstd = 1 / sqrt(ss / H + eps) as a pair rstd + lo, so that y = s (rstd + lo) w
// is off by little more than its last rounding (y decides the codes): the
// hardware's reciprocal root r0, good to about 22 bits, and one Newton step
// r0 (1 - ms r0^2) / 2 whose residual is exact to second order; ms = ss / H with
// its remainder.
__device__ __forceinline__ float root_pair(float ss, float h, float inv_h, float eps, float& lo) {
  const float q0 = ss * inv_h;
  const float ms = (isfinite(q0) ? fmaf(fmaf(-q0, h, ss), inv_h, q0) : q0) + eps;
  const float r0 = rsqrtf(ms);
  const float p = ms * r0;
  const float step = 0.5f * r0 * (fmaf(-p, r0, 1.0f) - fmaf(ms, r0, -p) * r0);
  const bool fine = isfinite(step);       // (not for ms = 0 or infinity)
  const float rstd = fine ? r0 + step : r0;
  lo = fine ? step - (rstd - r0) : 0.0f;
  return rstd;
}
// y of N elements in place of s
template <int N>
__device__ __forceinline__ void scale_row(float* y, const float* w, float rstd, float lo) {
  const f32x2 r2{rstd, rstd}, lo2{lo, lo};
#pragma unroll
  for (int j = 0; j < N; j += 2) {
    const f32x2 s2{y[j], y[j + 1]}, w2{w[j], w[j + 1]};
    const f32x2 t = mul2(s2, r2);
    const f32x2 e = fma2(s2, lo2, fma2(s2, r2, f32x2{-t.x, -t.y}));
    const f32x2 z = fma2(t, w2, mul2(e, w2));
    y[j] = z.x, y[j + 1] = z.y;
  }
}
// s = x + residual of N elements, and the sum of its squares
template <int N>
__device__ __forceinline__ void add_row(float* v, const float* u) {
#pragma unroll
  for (int j = 0; j < N; j += 2) {
    const f32x2 t = add2(f32x2{v[j], v[j + 1]}, f32x2{u[j], u[j + 1]});
    v[j] = t.x, v[j + 1] = t.y;
  }
}
template <int N>
__device__ __forceinline__ float square_sum(const float* v) {
  f32x2 sq{0.0f, 0.0f};
#pragma unroll
  for (int j = 0; j < N; j += 2) sq = fma2(f32x2{v[j], v[j + 1]}, f32x2{v[j], v[j + 1]}, sq);
  return sq.x + sq.y;
}

// The scale bytes of the rows that fill the last 128-row tile are zero. 16 bytes
// of a tile hold rows r, r + 32, r + 64 and r + 96, a word each.
__device__ __forceinline__ void zero_scale_rows(const NormArgs& a) {
  const int kb4 = a.H >> 7, live = static_cast<int>(a.T & 127);
  if (live == 0) return;
  uint8_t* tiles = a.scales + (a.T >> 7) * kb4 * 512;
  for (int i = blockIdx.x * blockDim.x + threadIdx.x; i < kb4 * 32; i += gridDim.x * blockDim.x) {
    const int r = i & 31;
    if (r >= live) {
      *(reinterpret_cast<uint4*>(tiles) + i) = make_uint4(0, 0, 0, 0);
    } else {
#pragma unroll
      for (int g = 1; g < 4; ++g)
        if (r + 32 * g >= live) *(reinterpret_cast<uint32_t*>(tiles) + 4 * i + g) = 0;
    }
  }
}

// an atomic only where it raises the value (which never falls)
__device__ __forceinline__ void raise_amax(const NormArgs& a, uint32_t amax) {
  unsigned int* const at = reinterpret_cast<unsigned int*>(a.amax);
  if (amax > *reinterpret_cast<volatile unsigned int*>(at)) atomicMax(at, amax);
}

// A CTA per row (few rows). SC: the mgq_scaling of the codes or kNoQuant; CH:
// 8-element chunks per thread.
template <int SC, int DT, int CH>
__global__ void __launch_bounds__(512, CH < 4 ? 2 : 1) norm_kernel(NormArgs a) {
  __shared__ float red[2][32];
  ptx::grid_wait();
  ptx::grid_launch();
  const int nchunk = a.H >> 3, stride = blockDim.x;
  const uint32_t lane = threadIdx.x & 31;
  const float h = static_cast<float>(a.H), inv_h = 1.0f / h;
  float ts = 1.0f;
  if (SC == MGQ_TENSOR_F32) ts = *a.ts;
  if (SC == MGQ_MX32_E8M0) zero_scale_rows(a);
  uint32_t amax = 0;
  int slot = 0;
  for (int64_t r = blockIdx.x; r < a.T; r += gridDim.x, slot ^= 1) {
    float v[CH][8], w[CH][8];
    float ss = 0.0f;
#pragma unroll
    for (int i = 0; i < CH; ++i) {
      const int c = threadIdx.x + i * stride;
      if (c < nchunk) {
        load_w8(a.w, a.wf32, c, w[i]);
        unpack8(*(reinterpret_cast<const uint4*>(a.x + r * a.H) + c), v[i]);
        if (a.res) {
          float u[8];
          unpack8(*(reinterpret_cast<const uint4*>(a.res + r * a.H) + c), u);
          add_row<8>(v[i], u);
        }
        if (a.sum) *(reinterpret_cast<uint4*>(a.sum + r * a.H) + c) = pack8(v[i]);
        ss += square_sum<8>(v[i]);
      }
    }
    bool none = false;
    ss = block_sum<false>(ss, red, slot, none);
    float lo;
    const float rstd = root_pair(ss, h, inv_h, a.eps, lo);
    if (a.rstd && threadIdx.x == 0) a.rstd[r] = rstd;
#pragma unroll
    for (int i = 0; i < CH; ++i) {
      const int c = threadIdx.x + i * stride;
      const bool in = c < nchunk;
      float* y = v[i];
      if (in) {
        scale_row<8>(y, w[i], rstd, lo);
        if (a.y) *(reinterpret_cast<uint4*>(a.y + r * a.H) + c) = pack8(y);
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) y[j] = 0.0f;
      }
      if (SC == kNoQuant) continue;
      uint32_t m = absmax<8>(y);
      float mult = ts;
      uint32_t sc = 0;
      float sinv = 0.0f;
      if (SC == MGQ_TENSOR_F32) {
        amax = max(amax, m);
      } else {
        m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, 1));
        m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, 2));
        if (SC == MGQ_MX32_E8M0) {
          mx_scale(m, FmtInfo<DT>::emax, a.rceil, sc, mult);
        } else {
          m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, 4));
          m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, 8));
          mult = blk_scale<DT>(m);
          sinv = __fdiv_rn(1.0f, mult);
        }
      }
      if (!in) continue;
      uint2 cw;
      cw.x = cvt_fp8x4_mul<DT>(y[0], y[1], y[2], y[3], mult);
      cw.y = cvt_fp8x4_mul<DT>(y[4], y[5], y[6], y[7], mult);
      *(reinterpret_cast<uint2*>(a.codes + r * a.H) + c) = cw;
      if (SC == MGQ_MX32_E8M0 && (lane & 3) == 0) a.scales[tiled_scale_offset(r, c >> 2, a.H >> 7)] = static_cast<uint8_t>(sc);
      if (SC == MGQ_BLK_1x128_F32 && (lane & 15) == 0)
        reinterpret_cast<float*>(a.scales)[static_cast<int64_t>(c >> 4) * a.T + r] = sinv;
    }
  }
  if (SC == MGQ_TENSOR_F32 && a.amax) {
    // one atomic a CTA
    amax = warp_max_u32(amax);
    uint32_t* const all = reinterpret_cast<uint32_t*>(red[slot]);
    if (lane == 0) all[threadIdx.x >> 5] = amax;
    __syncthreads();
    if (threadIdx.x < 32) {
      amax = warp_max_u32(lane < (blockDim.x + 31) >> 5 ? all[lane] : 0u);
      if (lane == 0) raise_amax(a, amax);
    }
  }
}

// 16 bf16 values of a lane, 32 bytes: one store where the row is 32-byte aligned
__device__ __forceinline__ void store16(uint16_t* p, const float* v, bool wide) {
  const uint4 a = pack8(v), b = pack8(v + 8);
  if (wide) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(a.x), "r"(a.y), "r"(a.z),
                 "r"(a.w), "r"(b.x), "r"(b.y), "r"(b.z), "r"(b.w)
                 : "memory");
  } else {
    reinterpret_cast<uint4*>(p)[0] = a;
    reinterpret_cast<uint4*>(p)[1] = b;
  }
}

// Many rows (H a multiple of 128). The instructions of a row that do not
// depend on its length (wait, reduction, root) are paid by every thread, so a
// thread takes U runs of 16 elements: two lanes hold an MX block, eight a 1x128
// block.
template <int SC, int DT, int U>
__global__ void __launch_bounds__(512) norm_stream_kernel(NormArgs a) {
  __shared__ __align__(16) float red[2][16];
  __shared__ uint64_t bars[kMaxSlots];
  extern __shared__ __align__(16) uint8_t ring_mem[];
  ptx::grid_wait();
  const int nrun = a.H >> 4, stride = blockDim.x, nw = blockDim.x >> 5;
  const uint32_t lane = threadIdx.x & 31;
  const float h = static_cast<float>(a.H), inv_h = 1.0f / h;
  float ts = 1.0f;
  if (SC == MGQ_TENSOR_F32) ts = *a.ts;
  RowRing<2> ring;
  const uint16_t* const src[2] = {a.x, a.res};
  ring.init(ring_mem, bars, a.ring, a.H * 2u);
  if (threadIdx.x == 0)
    for (int i = 0; i < a.ring.slots; ++i) ring.request(src, a.T);
  float w[U][16];
#pragma unroll
  for (int i = 0; i < U; ++i) {
    const int c = threadIdx.x + i * stride;
    if (c < nrun) {
      load_w8(a.w, a.wf32, 2 * c, w[i]);
      load_w8(a.w, a.wf32, 2 * c + 1, w[i] + 8);
    }
  }
  if (threadIdx.x < 32) (&red[0][0])[threadIdx.x] = 0.0f;
  __syncthreads();
  uint32_t amax = 0;
  int slot = 0;
  for (int64_t r = blockIdx.x; r < a.T; r += gridDim.x, slot ^= 1) {
    const bool here = ring.wait(a.ring.wait_ns);
    const uint4 *xr = ring.row(0), *rr = ring.row(1);
    const int64_t base = r * a.H;
    float v[U][16];
    float ss = 0.0f;
#pragma unroll
    for (int i = 0; i < U; ++i) {
      const int c = threadIdx.x + i * stride;
      if (c < nrun) {
        unpack8(xr[2 * c], v[i]);
        unpack8(xr[2 * c + 1], v[i] + 8);
        if (a.res) {
          float u[16];
          unpack8(rr[2 * c], u);
          unpack8(rr[2 * c + 1], u + 8);
          add_row<16>(v[i], u);
        }
        ss += square_sum<16>(v[i]);
      }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) ss += __shfl_xor_sync(0xFFFFFFFFu, ss, o);
    if (lane == 0) red[slot][threadIdx.x >> 5] = ss;
    if (__syncthreads_or(!here)) {
      report(a.ring.err, MGQ_ERR_TIMEOUT);
      ring.drain(a.ring.wait_ns);
      break;
    }
    ring.advance();                      // every thread has read the slot
    if (threadIdx.x == 0) ring.request(src, a.T);
    const float4* part = reinterpret_cast<const float4*>(red[slot]);
    float4 s4 = part[0];
    ss = (s4.x + s4.y) + (s4.z + s4.w);
    for (int i = 1; 4 * i < nw; ++i) {
      s4 = part[i];
      ss += (s4.x + s4.y) + (s4.z + s4.w);
    }
    float lo;
    const float rstd = root_pair(ss, h, inv_h, a.eps, lo);
    if (a.rstd && threadIdx.x == 0) a.rstd[r] = rstd;
    uint8_t* srow = SC == MGQ_MX32_E8M0 ? a.scales + tiled_scale_offset(r, 0, a.H >> 7) : nullptr;
#pragma unroll
    for (int i = 0; i < U; ++i) {
      const int c = threadIdx.x + i * stride;
      const bool in = c < nrun;          // (whole groups of eight lanes: H is a multiple of 128)
      float* y = v[i];
      if (in) {
        if (a.sum) store16(a.sum + base + 16 * c, y, a.wide);
        scale_row<16>(y, w[i], rstd, lo);
        if (a.y) store16(a.y + base + 16 * c, y, a.wide);
      }
      if (SC == kNoQuant) continue;
      uint32_t m = in ? absmax<16>(y) : 0u;
      float mult = ts;
      uint32_t sc = 0;
      float sinv = 0.0f;
      if (SC == MGQ_TENSOR_F32) {
        amax = max(amax, m);
      } else {
        m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, 1));
        if (SC == MGQ_MX32_E8M0) {
          mx_scale(m, FmtInfo<DT>::emax, a.rceil, sc, mult);
        } else {
          m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, 2));
          m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, 4));
          mult = blk_scale<DT>(m);
          sinv = __fdiv_rn(1.0f, mult);
        }
      }
      if (!in) continue;
      uint4 cw;
      cw.x = cvt_fp8x4_mul<DT>(y[0], y[1], y[2], y[3], mult);
      cw.y = cvt_fp8x4_mul<DT>(y[4], y[5], y[6], y[7], mult);
      cw.z = cvt_fp8x4_mul<DT>(y[8], y[9], y[10], y[11], mult);
      cw.w = cvt_fp8x4_mul<DT>(y[12], y[13], y[14], y[15], mult);
      *reinterpret_cast<uint4*>(a.codes + base + 16 * c) = cw;
      if (SC == MGQ_MX32_E8M0 && (lane & 1) == 0) srow[(c >> 3) * 512 + ((c >> 1) & 3)] = static_cast<uint8_t>(sc);
      if (SC == MGQ_BLK_1x128_F32 && (lane & 7) == 0)
        reinterpret_cast<float*>(a.scales)[static_cast<int64_t>(c >> 3) * a.T + r] = sinv;
    }
  }
  if (SC == MGQ_TENSOR_F32 && a.amax) {
    amax = warp_max_u32(amax);
    if (lane == 0) raise_amax(a, amax);
  }
  if (SC == MGQ_MX32_E8M0) zero_scale_rows(a);
}

// CTA size and chunks per thread for a row of `nchunk` 16-byte chunks.
void row_shape(int nchunk, int* threads, int* ch) {
  *ch = nchunk <= 256 ? 1 : nchunk <= 1024 ? 2 : 4;
  *threads = ((nchunk + *ch - 1) / *ch + 31) / 32 * 32;
}

constexpr int kNormThreads = 512;            // streamed forward: threads of an SM (twice that for many rows)
constexpr size_t kRingPerSm = 192 * 1024;    // shared memory for the rings of an SM's CTAs

// CTAs per SM and ring slots of a streamed kernel whose slot takes `slot`
// bytes: CTAs for `all` threads (at most 16), fewer where two slots each would
// not fit.
void ring_shape(int threads, int all, size_t slot, int* ctas, int* slots) {
  int n = all / threads;
  n = n < 1 ? 1 : n > 16 ? 16 : n;
  while (n > 1 && kRingPerSm / n < 2 * slot) --n;
  const int s = static_cast<int>(kRingPerSm / n / slot);
  *ctas = n;
  *slots = s < 2 ? 2 : s > kMaxSlots ? kMaxSlots : s;
}

// Allows the largest ring, once per device and kernel (attr_set: the launcher's):
// the limit is the function's, shared by all host threads, so a call never sets
// it to its own ring.
template <typename K>
bool allow_rings(K kern, bool (&attr_set)[64]) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return false;
  if (dev < 64 && attr_set[dev]) return true;
  if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(kRingPerSm)) != cudaSuccess)
    return false;
  if (dev < 64) attr_set[dev] = true;
  return true;
}

template <int SC, int DT, int U>
int launch_norm_stream(const NormArgs& a, int threads, int grid, size_t smem, cudaStream_t s) {
  auto kern = norm_stream_kernel<SC, DT, U>;
  static bool attr_set[64] = {false};
  if (!allow_rings(kern, attr_set)) return MGQ_ERR_CUDA;
  return launch_after(kern, dim3(grid), threads, smem, 1, s, a) ? MGQ_OK : MGQ_ERR_CUDA;
}

// Streamed once every CTA has two rows. Measured, MXFP8, direct / streamed, us:
// 1300 rows of 4096 9.7 / 8.8, 2500 of 2048 9.6 / 8.3, 5000 of 7168 64.9 / 54.4,
// 16384 of 4096 105 / 100; with less than two 700 of 2048 3.9 / 3.8, 1300 of
// 1024 3.6 / 4.3. Threads of an SM 256 / 512 / 1024: 5000 of 4096 32.7 / 31.9 /
// 32.9, 9000 of 1024 18.6 / 15.8 / 16.5; 1024 from nine rows a CTA on: 512 / 1024,
// 16384 of 4096 103 / 100, 9000 of 7168 100.5 / 96.7, eight rows (5000 of 5120)
// 40.2 / 41.2.
template <int SC, int DT>
int launch_norm(NormArgs a, cudaStream_t s) {
  if (a.H % 128 == 0) {
    const int u = a.H > 1024 ? 2 : 1, st = ((a.H / 16 + u - 1) / u + 31) / 32 * 32;
    const size_t slot = static_cast<size_t>(a.H) * 4;
    int ctas;
    ring_shape(st, 2 * kNormThreads, slot, &ctas, &a.ring.slots);
    if (a.T < static_cast<int64_t>(9) * num_sms() * ctas) ring_shape(st, kNormThreads, slot, &ctas, &a.ring.slots);
    const int64_t grid = static_cast<int64_t>(num_sms()) * ctas;
    if (a.T >= 2 * grid) {
      a.wide = ((reinterpret_cast<uintptr_t>(a.sum) | reinterpret_cast<uintptr_t>(a.y)) & 31) == 0;
      return u == 2 ? launch_norm_stream<SC, DT, 2>(a, st, static_cast<int>(grid), slot * a.ring.slots, s)
                    : launch_norm_stream<SC, DT, 1>(a, st, static_cast<int>(grid), slot * a.ring.slots, s);
    }
  }
  int threads, ch;
  row_shape(a.H >> 3, &threads, &ch);
  const int64_t most = static_cast<int64_t>(num_sms()) * (2048 / threads);
  const int grid = static_cast<int>(a.T < most ? a.T : most);
  auto kern = ch == 1 ? norm_kernel<SC, DT, 1> : ch == 2 ? norm_kernel<SC, DT, 2> : norm_kernel<SC, DT, 4>;
  return launch_after(kern, dim3(grid), threads, 0, 1, s, a) ? MGQ_OK : MGQ_ERR_CUDA;
}

struct NormBwdArgs {
  const uint16_t* dy;
  const uint16_t* s;
  const void* w;
  int wf32;
  const float* rstd;
  const uint16_t* dsum;   // or null
  int64_t T;
  int H;
  uint16_t* dx;
  float* part;            // [grid, H]
  RingArgs ring;
};

template <int CH, bool STREAM>
__global__ void __launch_bounds__(512) norm_bwd_kernel(NormBwdArgs a) {
  __shared__ float red[2][32];
  __shared__ uint64_t bars[kMaxSlots];
  extern __shared__ __align__(16) uint8_t ring_mem[];
  ptx::grid_wait();
  ptx::grid_launch();
  const int nchunk = a.H >> 3, stride = blockDim.x;
  const float inv_h = 1.0f / static_cast<float>(a.H);
  RowRing<3> ring;
  const uint16_t* const src[3] = {a.dy, a.s, a.dsum};
  if (STREAM) {
    ring.init(ring_mem, bars, a.ring, a.H * 2u);
    if (threadIdx.x == 0)
      for (int i = 0; i < a.ring.slots; ++i) ring.request(src, a.T);
  }
  float dw[CH][8], w[CH][8];
#pragma unroll
  for (int i = 0; i < CH; ++i) {
    if (static_cast<int>(threadIdx.x) + i * stride < nchunk) load_w8(a.w, a.wf32, threadIdx.x + i * stride, w[i]);
#pragma unroll
    for (int j = 0; j < 8; ++j) dw[i][j] = 0.0f;
  }
  int slot = 0;
  float rstd_next = blockIdx.x < a.T ? a.rstd[blockIdx.x] : 0.0f;
  for (int64_t r = blockIdx.x; r < a.T; r += gridDim.x, slot ^= 1) {
    const bool here = !STREAM || ring.wait(a.ring.wait_ns);
    const float rstd = rstd_next;
    if (r + gridDim.x < a.T) rstd_next = a.rstd[r + gridDim.x];
    const uint4* yr = STREAM ? ring.row(0) : reinterpret_cast<const uint4*>(a.dy + r * a.H);
    const uint4* sr = STREAM ? ring.row(1) : reinterpret_cast<const uint4*>(a.s + r * a.H);
    const uint4* dr = STREAM ? ring.row(2) : reinterpret_cast<const uint4*>(a.dsum + r * a.H);
    float g[CH][8], xh[CH][8];
    uint4 ds[CH];
    float c1 = 0.0f;
#pragma unroll
    for (int i = 0; i < CH; ++i) {
      const int c = threadIdx.x + i * stride;
      if (c < nchunk) {
        unpack8(yr[c], g[i]);
        unpack8(sr[c], xh[i]);
        if (a.dsum) ds[i] = dr[c];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          xh[i][j] *= rstd;
          dw[i][j] = fmaf(g[i][j], xh[i][j], dw[i][j]);
          g[i][j] *= w[i][j];
          c1 = fmaf(g[i][j], xh[i][j], c1);
        }
      }
    }
    bool lost = !here;
    c1 = block_sum<STREAM>(c1, red, slot, lost) * inv_h;
    if (STREAM) {
      if (lost) {
        report(a.ring.err, MGQ_ERR_TIMEOUT);
        ring.drain(a.ring.wait_ns);
        break;
      }
      ring.advance();
      if (threadIdx.x == 0) ring.request(src, a.T);
    }
#pragma unroll
    for (int i = 0; i < CH; ++i) {
      const int c = threadIdx.x + i * stride;
      if (c < nchunk) {
        float d[8];
        if (a.dsum) unpack8(ds[i], d);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float t = rstd * (g[i][j] - xh[i][j] * c1);
          d[j] = a.dsum ? t + d[j] : t;
        }
        *(reinterpret_cast<uint4*>(a.dx + r * a.H) + c) = pack8(d);
      }
    }
  }
#pragma unroll
  for (int i = 0; i < CH; ++i) {
    const int c = threadIdx.x + i * stride;
    if (c < nchunk) {
      float4* p = reinterpret_cast<float4*>(a.part + static_cast<int64_t>(blockIdx.x) * a.H) + 2 * c;
      p[0] = make_float4(dw[i][0], dw[i][1], dw[i][2], dw[i][3]);
      p[1] = make_float4(dw[i][4], dw[i][5], dw[i][6], dw[i][7]);
    }
  }
}

// dw[c] = beta dw[c] + the sum of the n partial rows, in a fixed order: each of
// the 32 warps of a CTA sums every 32nd row of 32 columns, kInFlight of them per
// trip to memory (measured 4, 8, 16: 1000 rows of 1024 6.4, 6.0, 6.0 us, 333 rows
// of 2048 5.9, 5.2, 5.5). Launched while the kernel above drains.
constexpr int kInFlight = 8;
__global__ void __launch_bounds__(1024) norm_dw_kernel(const float* part, int n, int H, float beta, float* dw) {
  __shared__ float sh[32][33];
  ptx::grid_wait();
  const int l = threadIdx.x & 31, c = blockIdx.x * 32 + l, w = threadIdx.x >> 5;
  float t = 0.0f;
  if (c < H) {
    const float* p = part + static_cast<int64_t>(w) * H + c;
    const int64_t step = static_cast<int64_t>(H) * 32;
    int r = w;
    for (; r + 32 * (kInFlight - 1) < n; r += 32 * kInFlight, p += kInFlight * step) {
      float v[kInFlight];
#pragma unroll
      for (int i = 0; i < kInFlight; ++i) v[i] = __ldcg(p + i * step);
#pragma unroll
      for (int o = kInFlight / 2; o > 0; o >>= 1)
#pragma unroll
        for (int i = 0; i < o; ++i) v[i] += v[i + o];
      t += v[0];
    }
    for (; r < n; r += 128, p += 4 * step) {
      float v[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] = r + 32 * i < n ? __ldcg(p + i * step) : 0.0f;
      t += (v[0] + v[1]) + (v[2] + v[3]);
    }
  }
  sh[w][l] = t;
  __syncthreads();
  // warp w sums column w of the 32 x 32 sums
  t = sh[l][w];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) t += __shfl_xor_sync(0xFFFFFFFFu, t, o);
  const int cw = blockIdx.x * 32 + w;
  if (l == 0 && cw < H) dw[cw] = beta == 0.0f ? t : fmaf(beta, dw[cw], t);
}

constexpr int64_t kMaxNormH = 16384;   // four chunks a thread of a 512-thread CTA

// Threads of an SM in the backward. 512, but 192 to 256 threads a row leave two
// rows to an SM then: four of 192 or three of 256 (9000 rows of 1408 28.6 / 22.4
// us, of 2048 32.1 / 28.0; more for other lengths costs them: 9000 rows of 4096
// 48.3 / 55.1, 4000 of 768 10.9 / 12.1).
int bwd_threads(int threads, int ch) {
  const int want = 4 * threads < 768 ? 4 * threads : 768;
  return ch == 1 && want > 512 ? want : 512;
}

// rows of partial sums of the backward for T rows of H elements: its grid
int bwd_grid(int64_t T, int64_t H) {
  int threads, ch, ctas, slots;
  row_shape(static_cast<int>(H >> 3), &threads, &ch);
  ring_shape(threads, bwd_threads(threads, ch), static_cast<size_t>(H) * 6, &ctas, &slots);
  const int64_t g = static_cast<int64_t>(num_sms()) * ctas;
  return static_cast<int>(T < g ? T : g);
}

template <int CH>
int launch_bwd(NormBwdArgs a, int threads, int grid, cudaStream_t s) {
  const size_t slot = static_cast<size_t>(a.H) * 6;
  int ctas;
  ring_shape(threads, bwd_threads(threads, CH), slot, &ctas, &a.ring.slots);
  // Streamed from 1.5 rows a CTA on (direct / streamed, us: 600 rows of 4096 9.9 /
  // 8.9, 16384 of 4096 123 / 80; 600 of 2048, 1.3 a CTA, 6.3 / 6.5). Four chunks a
  // thread beside the ring do not fit the registers.
  if constexpr (CH < 4) {
    if (2 * a.T > 3 * static_cast<int64_t>(grid)) {
      auto kern = norm_bwd_kernel<CH, true>;
      static bool attr_set[64] = {false};
      if (!allow_rings(kern, attr_set)) return MGQ_ERR_CUDA;
      return launch_after(kern, dim3(grid), threads, slot * a.ring.slots, 1, s, a) ? MGQ_OK : MGQ_ERR_CUDA;
    }
  }
  return launch_after(norm_bwd_kernel<CH, false>, dim3(grid), threads, 0, 1, s, a) ? MGQ_OK : MGQ_ERR_CUDA;
}

void ring_limits(RingArgs& a) {
  debug_knobs(&a.stall, &a.wait_ns);
  a.err = error_word();
}

bool norm_sizes_ok(int64_t T, int64_t H) {
  return T >= 0 && T <= (int64_t(1) << 40) && H >= 8 && H % 8 == 0 && H <= kMaxNormH;
}

}  // namespace
}  // namespace mgq

using namespace mgq;

extern "C" int mgq_add_rmsnorm_quantize(const void* x_bf16, const void* residual_bf16, const void* w, int w_dtype,
                                        int64_t T, int64_t H, float eps, void* sum_bf16, void* y_bf16,
                                        const mgq_qdesc* q, float* rstd, void* stream) {
  MGQ_CHECK_ARG(norm_sizes_ok(T, H));
  MGQ_CHECK_ARG(w_dtype == MGQ_OUT_BF16 || w_dtype == MGQ_OUT_F32);
  MGQ_CHECK_ARG(eps >= 0.0f);
  if (q) {
    if (q->dtype != MGQ_E4M3 && q->dtype != MGQ_E5M2) return MGQ_ERR_UNSUPPORTED;
    if (q->scaling != MGQ_MX32_E8M0 && q->scaling != MGQ_BLK_1x128_F32 && q->scaling != MGQ_TENSOR_F32)
      return MGQ_ERR_UNSUPPORTED;
    if (q->col.data) return MGQ_ERR_UNSUPPORTED;
    MGQ_CHECK_ARG(H % 128 == 0);
    if (q->scaling == MGQ_MX32_E8M0) MGQ_CHECK_ARG(q->e8m0_mode == MGQ_E8M0_RCEIL || q->e8m0_mode == MGQ_E8M0_FLOOR);
  }
  if (T == 0) return MGQ_OK;
  MGQ_CHECK_ARG(sum_bf16 || y_bf16 || q || rstd);
  MGQ_CHECK_ARG(x_bf16 && w && aligned16(x_bf16) && aligned16(residual_bf16) && aligned16(w) &&
                aligned16(sum_bf16) && aligned16(y_bf16));
  if (q) {
    MGQ_CHECK_ARG(q->row.data && aligned16(q->row.data) && aligned16(q->row.scale));
    MGQ_CHECK_ARG(q->scaling == MGQ_TENSOR_F32 ? q->tensor_scale != nullptr : q->row.scale != nullptr);
  }
  NormArgs a{};
  a.x = static_cast<const uint16_t*>(x_bf16);
  a.res = static_cast<const uint16_t*>(residual_bf16);
  a.w = w;
  a.wf32 = w_dtype == MGQ_OUT_F32;
  a.T = T;
  a.H = static_cast<int>(H);
  a.eps = eps;
  a.sum = static_cast<uint16_t*>(sum_bf16);
  a.y = static_cast<uint16_t*>(y_bf16);
  a.rstd = rstd;
  ring_limits(a.ring);
  cudaStream_t s = as_stream(stream);
  if (!q) return launch_norm<kNoQuant, MGQ_E4M3>(a, s);
  {
    a.codes = static_cast<uint8_t*>(q->row.data);
    a.scales = static_cast<uint8_t*>(q->row.scale);
    a.ts = q->tensor_scale;
    a.amax = q->amax_out;
    a.rceil = q->e8m0_mode == MGQ_E8M0_RCEIL;
    const bool e4 = q->dtype == MGQ_E4M3;
    if (q->scaling == MGQ_MX32_E8M0)
      return e4 ? launch_norm<MGQ_MX32_E8M0, MGQ_E4M3>(a, s) : launch_norm<MGQ_MX32_E8M0, MGQ_E5M2>(a, s);
    if (q->scaling == MGQ_BLK_1x128_F32)
      return e4 ? launch_norm<MGQ_BLK_1x128_F32, MGQ_E4M3>(a, s) : launch_norm<MGQ_BLK_1x128_F32, MGQ_E5M2>(a, s);
    return e4 ? launch_norm<MGQ_TENSOR_F32, MGQ_E4M3>(a, s) : launch_norm<MGQ_TENSOR_F32, MGQ_E5M2>(a, s);
  }
}

extern "C" size_t mgq_add_rmsnorm_bwd_workspace_size(int64_t T, int64_t H) {
  if (!norm_sizes_ok(T, H)) return 0;
  return static_cast<size_t>(bwd_grid(T, H)) * static_cast<size_t>(H) * sizeof(float);
}

extern "C" int mgq_add_rmsnorm_bwd(const void* dy_bf16, const void* s_bf16, const void* w, int w_dtype,
                                   const float* rstd, const void* dsum_bf16, int64_t T, int64_t H, void* dx_bf16,
                                   float* dw, float beta, void* workspace, size_t ws_bytes, void* stream) {
  MGQ_CHECK_ARG(norm_sizes_ok(T, H));
  MGQ_CHECK_ARG(w_dtype == MGQ_OUT_BF16 || w_dtype == MGQ_OUT_F32);
  MGQ_CHECK_ARG(dw);
  if (T > 0) {
    MGQ_CHECK_ARG(dy_bf16 && s_bf16 && w && rstd && dx_bf16 && workspace);
    MGQ_CHECK_ARG(aligned16(dy_bf16) && aligned16(s_bf16) && aligned16(w) && aligned16(dsum_bf16) &&
                  aligned16(dx_bf16) && aligned16(workspace));
    MGQ_CHECK_ARG(ws_bytes >= mgq_add_rmsnorm_bwd_workspace_size(T, H));
  }
  cudaStream_t s = as_stream(stream);
  NormBwdArgs a{};
  a.dy = static_cast<const uint16_t*>(dy_bf16);
  a.s = static_cast<const uint16_t*>(s_bf16);
  a.w = w;
  a.wf32 = w_dtype == MGQ_OUT_F32;
  a.rstd = rstd;
  a.dsum = static_cast<const uint16_t*>(dsum_bf16);
  a.T = T;
  a.H = static_cast<int>(H);
  a.dx = static_cast<uint16_t*>(dx_bf16);
  a.part = static_cast<float*>(workspace);
  ring_limits(a.ring);
  const int grid = bwd_grid(T, H);
  if (T > 0) {
    int threads, ch;
    row_shape(a.H >> 3, &threads, &ch);
    const int rc = ch == 1 ? launch_bwd<1>(a, threads, grid, s) : ch == 2 ? launch_bwd<2>(a, threads, grid, s)
                                                                          : launch_bwd<4>(a, threads, grid, s);
    if (rc != MGQ_OK) return rc;
  }
  return launch_after(norm_dw_kernel, dim3((a.H + 31) / 32), 1024, 0, 1, s, static_cast<const float*>(a.part), grid, a.H,
                      beta, dw)
             ? MGQ_OK
             : MGQ_ERR_CUDA;
}
