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

// the weight chunk c (8 values) as float32; wf32 selects float32 storage
__device__ __forceinline__ void load_w8(const void* w, bool wf32, int c, float* v) {
  if (wf32) {
    const float4* p = reinterpret_cast<const float4*>(w) + 2 * c;
    const float4 a = __ldg(p), b = __ldg(p + 1);
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
    v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
  } else {
    unpack8(__ldg(reinterpret_cast<const uint4*>(w) + c), v);
  }
}

// max |v| with NaN winning, as float bits
__device__ __forceinline__ uint32_t absmax8(const float* v) {
  float m = 0.0f;
#pragma unroll
  for (int j = 0; j < 8; ++j) asm("max.NaN.f32 %0, %0, %1;" : "+f"(m) : "f"(fabsf(v[j])));
  return __float_as_uint(m);
}

// Sum over the CTA; `slot` alternates between two shared arrays from one call
// to the next, so that one barrier a call is enough.
__device__ __forceinline__ float block_sum(float v, float (*red)[32], int slot) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
  const int warp = threadIdx.x >> 5, nw = blockDim.x >> 5;
  if (nw == 1) {
    __syncwarp();
    return v;
  }
  if ((threadIdx.x & 31) == 0) red[slot][warp] = v;
  __syncthreads();
  float t = (threadIdx.x & 31) < nw ? red[slot][threadIdx.x & 31] : 0.0f;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) t += __shfl_xor_sync(0xFFFFFFFFu, t, o);
  return t;
}

constexpr int kMaxSlots = 8;
constexpr uint64_t kWaitNs = 2000000000ull;   // limit of a wait for a row's copies

// A ring of row slots filled by bulk copies: NS source rows side by side per
// slot. Thread 0 requests; the barrier that every reduction passes frees a slot.
template <int NS>
struct RowRing {
  uint64_t* full;
  uint8_t* mem;
  uint32_t row_bytes;
  int slots, st, ask;      // slot to read next, slot to fill next
  uint32_t ph;
  int64_t next;            // row to request next

  __device__ __forceinline__ void init(uint8_t* base, uint64_t* bars, int n, uint32_t bytes) {
    full = bars;
    mem = base;
    row_bytes = bytes;
    slots = n;
    st = ask = 0;
    ph = 0;
    next = blockIdx.x;
    if (threadIdx.x == 0) {
      for (int i = 0; i < n; ++i) ptx::mbar_init(&full[i], 1);
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
  __device__ __forceinline__ bool wait() { return ptx::mbar_wait(&full[st], ph, kWaitNs); }
  __device__ __forceinline__ const uint4* row(int i) const {
    return reinterpret_cast<const uint4*>(mem + (static_cast<size_t>(st) * NS + i) * row_bytes);
  }
  // after a wait that ran out: give the copies in flight a last, short chance
  __device__ __forceinline__ void drain() {
    for (int i = 0; i < slots && threadIdx.x == 0; ++i)
      ptx::mbar_wait(&full[(st + i) % slots], ph ^ (st + i >= slots ? 1u : 0u), kWaitNs / 100);
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
  int slots;             // streamed: ring slots
  int* err;
};

// SC: the mgq_scaling of the codes or kNoQuant; CH: chunks per thread; STREAM:
// rows through the ring
template <int SC, int DT, int CH, bool STREAM>
__global__ void __launch_bounds__(512) norm_kernel(NormArgs a) {
  __shared__ float red[2][32];
  __shared__ uint64_t bars[kMaxSlots];
  extern __shared__ __align__(16) uint8_t ring_mem[];
  const int nchunk = a.H >> 3, stride = blockDim.x;
  const uint32_t lane = threadIdx.x & 31;
  float ts = 1.0f;
  if (SC == MGQ_TENSOR_F32) ts = __ldg(a.ts);
  RowRing<2> ring;
  const uint16_t* const src[2] = {a.x, a.res};
  if (STREAM) {
    ring.init(ring_mem, bars, a.slots, a.H * 2u);
    if (threadIdx.x == 0)
      for (int i = 0; i < a.slots; ++i) ring.request(src, a.T);
  }
  float w[CH][8];
  if (STREAM) {
#pragma unroll
    for (int i = 0; i < CH; ++i)
      if (static_cast<int>(threadIdx.x) + i * stride < nchunk) load_w8(a.w, a.wf32, threadIdx.x + i * stride, w[i]);
  }
  uint32_t amax = 0;
  int slot = 0;
  for (int64_t r = blockIdx.x; r < a.T; r += gridDim.x, slot ^= 1) {
    if (STREAM && !ring.wait()) {
      report(a.err, MGQ_ERR_TIMEOUT);
      ring.drain();
      break;
    }
    const uint4* xr = STREAM ? ring.row(0) : reinterpret_cast<const uint4*>(a.x + r * a.H);
    const uint4* rr = STREAM ? ring.row(1) : reinterpret_cast<const uint4*>(a.res + r * a.H);
    float v[CH][8];
    float ss = 0.0f;
#pragma unroll
    for (int i = 0; i < CH; ++i) {
      const int c = threadIdx.x + i * stride;
      if (c < nchunk) {
        if (!STREAM) load_w8(a.w, a.wf32, c, w[i]);
        unpack8(xr[c], v[i]);
        if (a.res) {
          float u[8];
          unpack8(rr[c], u);
#pragma unroll
          for (int j = 0; j < 8; j += 2) {
            const f32x2 t = add2(f32x2{v[i][j], v[i][j + 1]}, f32x2{u[j], u[j + 1]});
            v[i][j] = t.x, v[i][j + 1] = t.y;
          }
        }
        if (a.sum) *(reinterpret_cast<uint4*>(a.sum + r * a.H) + c) = pack8(v[i]);
        f32x2 sq{0.0f, 0.0f};
#pragma unroll
        for (int j = 0; j < 8; j += 2) {
          const f32x2 t{v[i][j], v[i][j + 1]};
          sq = fma2(t, t, sq);
        }
        ss += sq.x + sq.y;
      }
    }
    ss = block_sum(ss, red, slot);
    if (STREAM) {
      ring.advance();                      // every thread has read the slot
      if (threadIdx.x == 0) ring.request(src, a.T);
    }
    // rstd as a pair rstd + lo (lo: one Newton step's correction), so that y
    // below is off by little more than its last rounding: y decides the codes
    const float ms = __fadd_rn(__fdiv_rn(ss, static_cast<float>(a.H)), a.eps);
    const float rstd = __fdiv_rn(1.0f, __fsqrt_rn(ms));
    const float p = __fmul_rn(ms, rstd);
    float lo = 0.5f * rstd * (fmaf(-p, rstd, 1.0f) - __fmul_rn(fmaf(ms, rstd, -p), rstd));
    if (!isfinite(lo)) lo = 0.0f;
    if (a.rstd && threadIdx.x == 0) a.rstd[r] = rstd;
#pragma unroll
    for (int i = 0; i < CH; ++i) {
      const int c = threadIdx.x + i * stride;
      const bool in = c < nchunk;
      float* y = v[i];
      if (in) {
#pragma unroll
        for (int j = 0; j < 8; j += 2) {
          const f32x2 s2{y[j], y[j + 1]}, w2{w[i][j], w[i][j + 1]}, r2{rstd, rstd}, lo2{lo, lo};
          const f32x2 t = mul2(s2, r2);
          const f32x2 e = fma2(s2, lo2, fma2(s2, r2, f32x2{-t.x, -t.y}));
          const f32x2 z = fma2(t, w2, mul2(e, w2));
          y[j] = z.x, y[j + 1] = z.y;
        }
        if (a.y) *(reinterpret_cast<uint4*>(a.y + r * a.H) + c) = pack8(y);
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) y[j] = 0.0f;
      }
      if (SC == kNoQuant) continue;
      uint32_t m = absmax8(y);
      float mult = ts;
      uint32_t word = 0;
      float sinv = 0.0f;
      if (SC == MGQ_TENSOR_F32) {
        amax = max(amax, m);
      } else {
        m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, 1));
        m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, 2));
        if (SC == MGQ_MX32_E8M0) {
          const int e = mx_exponent(m, FmtInfo<DT>::emax, a.rceil != 0);
          mult = mx_multiplier(e);
          // the four blocks' scale bytes of these 128 elements, in lane 16 j
          const uint32_t sc = mx_scale_code(e);
          word = sc | (__shfl_down_sync(0xFFFFFFFFu, sc, 4) << 8) | (__shfl_down_sync(0xFFFFFFFFu, sc, 8) << 16) |
                 (__shfl_down_sync(0xFFFFFFFFu, sc, 12) << 24);
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
      if (SC == MGQ_MX32_E8M0 && (lane & 15) == 0)
        *reinterpret_cast<uint32_t*>(a.scales + tiled_scale_offset(r, c >> 2, a.H >> 7)) = word;
      if (SC == MGQ_BLK_1x128_F32 && (lane & 15) == 0)
        reinterpret_cast<float*>(a.scales)[static_cast<int64_t>(c >> 4) * a.T + r] = sinv;
    }
  }
  if (SC == MGQ_TENSOR_F32 && a.amax) {
    amax = warp_max_u32(amax);
    if (lane == 0 && amax) atomicMax(reinterpret_cast<unsigned int*>(a.amax), amax);
  }
  // the scale bytes of the rows that fill the last 128-row tile are zero
  if (SC == MGQ_MX32_E8M0) {
    const int kb4 = a.H >> 7, rest = static_cast<int>((128 - (a.T & 127)) & 127) * kb4;
    for (int i = blockIdx.x * stride + threadIdx.x; i < rest; i += gridDim.x * stride)
      *reinterpret_cast<uint32_t*>(a.scales + tiled_scale_offset(a.T + i / kb4, 4 * (i % kb4), kb4)) = 0;
  }
}

// CTA size and chunks per thread for a row of `nchunk` 16-byte chunks.
void row_shape(int nchunk, int* threads, int* ch) {
  *ch = nchunk <= 256 ? 1 : nchunk <= 1024 ? 2 : 4;
  *threads = ((nchunk + *ch - 1) / *ch + 31) / 32 * 32;
}

constexpr int kNormThreads = 1024, kNormBwdThreads = 512;   // streamed: threads of an SM
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

template <typename K>
bool allow_smem(K kern, size_t bytes) {
  return cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(bytes)) == cudaSuccess;
}

template <int SC, int DT, int CH>
int launch_norm_ch(NormArgs a, int threads, cudaStream_t s) {
  const size_t slot = static_cast<size_t>(a.H) * 4;
  int ctas;
  ring_shape(threads, kNormThreads, slot, &ctas, &a.slots);
  const int64_t grid = static_cast<int64_t>(num_sms()) * ctas;
  if (a.T >= 4 * grid) {
    auto kern = norm_kernel<SC, DT, CH, true>;
    const size_t smem = slot * a.slots;
    if (!allow_smem(kern, smem)) return MGQ_ERR_CUDA;
    kern<<<static_cast<int>(grid), threads, smem, s>>>(a);
  } else {
    const int64_t most = static_cast<int64_t>(num_sms()) * (2048 / threads);
    norm_kernel<SC, DT, CH, false><<<static_cast<int>(a.T < most ? a.T : most), threads, 0, s>>>(a);
  }
  MGQ_LAUNCH_CHECK();
  return MGQ_OK;
}

template <int SC, int DT>
int launch_norm(const NormArgs& a, cudaStream_t s) {
  int threads, ch;
  row_shape(a.H >> 3, &threads, &ch);
  return ch == 1 ? launch_norm_ch<SC, DT, 1>(a, threads, s) : ch == 2 ? launch_norm_ch<SC, DT, 2>(a, threads, s)
                                                                      : launch_norm_ch<SC, DT, 4>(a, threads, s);
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
  int slots;
  int* err;
};

template <int CH, bool STREAM>
__global__ void __launch_bounds__(512) norm_bwd_kernel(NormBwdArgs a) {
  __shared__ float red[2][32];
  __shared__ uint64_t bars[kMaxSlots];
  extern __shared__ __align__(16) uint8_t ring_mem[];
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int nchunk = a.H >> 3, stride = blockDim.x;
  const float inv_h = 1.0f / static_cast<float>(a.H);
  RowRing<3> ring;
  const uint16_t* const src[3] = {a.dy, a.s, a.dsum};
  if (STREAM) {
    ring.init(ring_mem, bars, a.slots, a.H * 2u);
    if (threadIdx.x == 0)
      for (int i = 0; i < a.slots; ++i) ring.request(src, a.T);
  }
  float dw[CH][8], w[CH][8];
#pragma unroll
  for (int i = 0; i < CH; ++i) {
    if (static_cast<int>(threadIdx.x) + i * stride < nchunk) load_w8(a.w, a.wf32, threadIdx.x + i * stride, w[i]);
#pragma unroll
    for (int j = 0; j < 8; ++j) dw[i][j] = 0.0f;
  }
  int slot = 0;
  float rstd_next = blockIdx.x < a.T ? __ldg(a.rstd + blockIdx.x) : 0.0f;
  for (int64_t r = blockIdx.x; r < a.T; r += gridDim.x, slot ^= 1) {
    if (STREAM && !ring.wait()) {
      report(a.err, MGQ_ERR_TIMEOUT);
      ring.drain();
      break;
    }
    const float rstd = rstd_next;
    if (r + gridDim.x < a.T) rstd_next = __ldg(a.rstd + r + gridDim.x);
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
    c1 = block_sum(c1, red, slot) * inv_h;
    if (STREAM) {
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
// the 32 warps of a CTA sums every 32nd row of 32 columns, four in flight.
// Launched while the kernel above drains.
__global__ void __launch_bounds__(1024) norm_dw_kernel(const float* part, int n, int H, float beta, float* dw) {
  __shared__ float sh[32][33];
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int l = threadIdx.x & 31, c = blockIdx.x * 32 + l, w = threadIdx.x >> 5;
  float t = 0.0f;
  if (c < H) {
    for (int r = w; r < n; r += 128) {
      float v[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] = r + 32 * i < n ? part[static_cast<int64_t>(r + 32 * i) * H + c] : 0.0f;
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

// rows of partial sums of the backward for T rows of H elements: its grid
int bwd_grid(int64_t T, int64_t H) {
  int threads, ch, ctas, slots;
  row_shape(static_cast<int>(H >> 3), &threads, &ch);
  ring_shape(threads, kNormBwdThreads, static_cast<size_t>(H) * 6, &ctas, &slots);
  const int64_t g = static_cast<int64_t>(num_sms()) * ctas;
  return static_cast<int>(T < g ? T : g);
}

template <int CH>
int launch_bwd(NormBwdArgs a, int threads, int grid, cudaStream_t s) {
  const size_t slot = static_cast<size_t>(a.H) * 6;
  int ctas;
  ring_shape(threads, kNormBwdThreads, slot, &ctas, &a.slots);
  // (four chunks a thread beside the ring do not fit the registers)
  if constexpr (CH < 4) {
    if (a.T >= 2 * static_cast<int64_t>(grid)) {
      auto kern = norm_bwd_kernel<CH, true>;
      const size_t smem = slot * a.slots;
      if (!allow_smem(kern, smem)) return MGQ_ERR_CUDA;
      kern<<<grid, threads, smem, s>>>(a);
      MGQ_LAUNCH_CHECK();
      return MGQ_OK;
    }
  }
  norm_bwd_kernel<CH, false><<<grid, threads, 0, s>>>(a);
  MGQ_LAUNCH_CHECK();
  return MGQ_OK;
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
  a.err = error_word();
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
  a.err = error_word();
  const int grid = bwd_grid(T, H);
  if (T > 0) {
    int threads, ch;
    row_shape(a.H >> 3, &threads, &ch);
    const int rc = ch == 1 ? launch_bwd<1>(a, threads, grid, s) : ch == 2 ? launch_bwd<2>(a, threads, grid, s)
                                                                          : launch_bwd<4>(a, threads, grid, s);
    if (rc != MGQ_OK) return rc;
  }
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = T > 0 ? 1 : 0;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((a.H + 31) / 32);
  cfg.blockDim = dim3(1024);
  cfg.stream = s;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  if (cudaLaunchKernelEx(&cfg, norm_dw_kernel, static_cast<const float*>(a.part), grid, a.H, beta, dw) != cudaSuccess) {
    (void)cudaGetLastError();
    return MGQ_ERR_CUDA;
  }
  return MGQ_OK;
}
