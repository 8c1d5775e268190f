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
#include "mgq_internal.h"
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

// Sum over the CTA; `slot` alternates between two shared arrays from one call
// to the next, so that one barrier a call is enough.
__device__ __forceinline__ float block_sum(float v, float (*red)[32], int slot) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
  const int warp = threadIdx.x >> 5, nw = blockDim.x >> 5;
  if (nw == 1) return v;
  if ((threadIdx.x & 31) == 0) red[slot][warp] = v;
  __syncthreads();
  float t = (threadIdx.x & 31) < nw ? red[slot][threadIdx.x & 31] : 0.0f;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) t += __shfl_xor_sync(0xFFFFFFFFu, t, o);
  return t;
}

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
};

// SC: the mgq_scaling of the codes or kNoQuant; CH: chunks per thread
template <int SC, int DT, int CH>
__global__ void __launch_bounds__(512) norm_kernel(NormArgs a) {
  __shared__ float red[2][32];
  const int nchunk = a.H >> 3, stride = blockDim.x;
  const uint32_t lane = threadIdx.x & 31;
  const float inv_h = 1.0f / static_cast<float>(a.H);
  float ts = 1.0f;
  if (SC == MGQ_TENSOR_F32) ts = __ldg(a.ts);
  uint32_t amax = 0;
  int slot = 0;
  for (int64_t r = blockIdx.x; r < a.T; r += gridDim.x, slot ^= 1) {
    float v[CH][8];
    float ss = 0.0f;
#pragma unroll
    for (int i = 0; i < CH; ++i) {
      const int c = threadIdx.x + i * stride;
      if (c < nchunk) {
        unpack8(*(reinterpret_cast<const uint4*>(a.x + r * a.H) + c), v[i]);
        if (a.res) {
          float u[8];
          unpack8(*(reinterpret_cast<const uint4*>(a.res + r * a.H) + c), u);
#pragma unroll
          for (int j = 0; j < 8; ++j) v[i][j] += u[j];
        }
        if (a.sum) *(reinterpret_cast<uint4*>(a.sum + r * a.H) + c) = pack8(v[i]);
#pragma unroll
        for (int j = 0; j < 8; ++j) ss = fmaf(v[i][j], v[i][j], ss);
      }
    }
    ss = block_sum(ss, red, slot);
    const float rstd = 1.0f / sqrtf(fmaf(ss, inv_h, a.eps));
    if (a.rstd && threadIdx.x == 0) a.rstd[r] = rstd;
#pragma unroll
    for (int i = 0; i < CH; ++i) {
      const int c = threadIdx.x + i * stride;
      const bool in = c < nchunk;
      float* y = v[i];
      if (in) {
        float w[8];
        load_w8(a.w, a.wf32, c, w);
#pragma unroll
        for (int j = 0; j < 8; ++j) y[j] = y[j] * rstd * w[j];
        if (a.y) *(reinterpret_cast<uint4*>(a.y + r * a.H) + c) = pack8(y);
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) y[j] = 0.0f;
      }
      if (SC == kNoQuant) continue;
      uint32_t m = absmax_bits_f32(y, 8);
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
    const int64_t rp = (a.T + 127) / 128 * 128;
    for (int64_t r = a.T + blockIdx.x; r < rp; r += gridDim.x)
      for (int b = threadIdx.x; b < (a.H >> 7); b += stride)
        *reinterpret_cast<uint32_t*>(a.scales + tiled_scale_offset(r, 4 * b, a.H >> 7)) = 0;
  }
}

// CTA size and chunks per thread for a row of `nchunk` 16-byte chunks.
void row_shape(int nchunk, int* threads, int* ch) {
  *ch = nchunk <= 512 ? 1 : nchunk <= 1024 ? 2 : 4;
  *threads = ((nchunk + *ch - 1) / *ch + 31) / 32 * 32;
}

template <int SC, int DT>
void launch_norm(const NormArgs& a, cudaStream_t s) {
  int threads, ch;
  row_shape(a.H >> 3, &threads, &ch);
  const int64_t per_sm = 2048 / threads;
  const int grid = static_cast<int>(a.T < num_sms() * per_sm ? a.T : num_sms() * per_sm);
  if (ch == 1) norm_kernel<SC, DT, 1><<<grid, threads, 0, s>>>(a);
  else if (ch == 2) norm_kernel<SC, DT, 2><<<grid, threads, 0, s>>>(a);
  else norm_kernel<SC, DT, 4><<<grid, threads, 0, s>>>(a);
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
};

template <int CH>
__global__ void __launch_bounds__(512) norm_bwd_kernel(NormBwdArgs a) {
  __shared__ float red[2][32];
  const int nchunk = a.H >> 3, stride = blockDim.x;
  const float inv_h = 1.0f / static_cast<float>(a.H);
  float dw[CH][8];
#pragma unroll
  for (int i = 0; i < CH; ++i)
#pragma unroll
    for (int j = 0; j < 8; ++j) dw[i][j] = 0.0f;
  int slot = 0;
  for (int64_t r = blockIdx.x; r < a.T; r += gridDim.x, slot ^= 1) {
    float g[CH][8], xh[CH][8];
    const float rstd = __ldg(a.rstd + r);
    float c1 = 0.0f;
#pragma unroll
    for (int i = 0; i < CH; ++i) {
      const int c = threadIdx.x + i * stride;
      if (c < nchunk) {
        float w[8];
        unpack8(__ldg(reinterpret_cast<const uint4*>(a.dy + r * a.H) + c), g[i]);
        unpack8(__ldg(reinterpret_cast<const uint4*>(a.s + r * a.H) + c), xh[i]);
        load_w8(a.w, a.wf32, c, w);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          xh[i][j] *= rstd;
          dw[i][j] = fmaf(g[i][j], xh[i][j], dw[i][j]);
          g[i][j] *= w[j];
          c1 = fmaf(g[i][j], xh[i][j], c1);
        }
      }
    }
    c1 = block_sum(c1, red, slot) * inv_h;
#pragma unroll
    for (int i = 0; i < CH; ++i) {
      const int c = threadIdx.x + i * stride;
      if (c < nchunk) {
        float d[8];
        if (a.dsum) unpack8(*(reinterpret_cast<const uint4*>(a.dsum + r * a.H) + c), d);
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
// the 8 warps of a CTA sums every eighth row of 32 columns.
__global__ void __launch_bounds__(256) norm_dw_kernel(const float* part, int n, int H, float beta, float* dw) {
  __shared__ float sh[8][33];
  const int c = blockIdx.x * 32 + (threadIdx.x & 31), w = threadIdx.x >> 5;
  float t = 0.0f;
  if (c < H)
    for (int r = w; r < n; r += 8) t += part[static_cast<int64_t>(r) * H + c];
  sh[w][threadIdx.x & 31] = t;
  __syncthreads();
  if (w == 0 && c < H) {
    t = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) t += sh[i][threadIdx.x];
    dw[c] = beta == 0.0f ? t : fmaf(beta, dw[c], t);
  }
}

constexpr int64_t kMaxNormH = 16384;   // four chunks a thread of a 512-thread CTA

// rows of partial sums of the backward for T rows of H elements
int bwd_grid(int64_t T, int64_t H) {
  int threads, ch;
  row_shape(static_cast<int>(H >> 3), &threads, &ch);
  const int64_t g = static_cast<int64_t>(num_sms()) * (1024 / threads > 8 ? 8 : 1024 / threads);
  return static_cast<int>(T < g ? T : g);
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
  cudaStream_t s = as_stream(stream);
  if (!q) {
    launch_norm<kNoQuant, MGQ_E4M3>(a, s);
  } else {
    a.codes = static_cast<uint8_t*>(q->row.data);
    a.scales = static_cast<uint8_t*>(q->row.scale);
    a.ts = q->tensor_scale;
    a.amax = q->amax_out;
    a.rceil = q->e8m0_mode == MGQ_E8M0_RCEIL;
    const bool e4 = q->dtype == MGQ_E4M3;
    if (q->scaling == MGQ_MX32_E8M0)
      e4 ? launch_norm<MGQ_MX32_E8M0, MGQ_E4M3>(a, s) : launch_norm<MGQ_MX32_E8M0, MGQ_E5M2>(a, s);
    else if (q->scaling == MGQ_BLK_1x128_F32)
      e4 ? launch_norm<MGQ_BLK_1x128_F32, MGQ_E4M3>(a, s) : launch_norm<MGQ_BLK_1x128_F32, MGQ_E5M2>(a, s);
    else
      e4 ? launch_norm<MGQ_TENSOR_F32, MGQ_E4M3>(a, s) : launch_norm<MGQ_TENSOR_F32, MGQ_E5M2>(a, s);
  }
  MGQ_LAUNCH_CHECK();
  return MGQ_OK;
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
  const int grid = bwd_grid(T, H);
  if (T > 0) {
    int threads, ch;
    row_shape(a.H >> 3, &threads, &ch);
    if (ch == 1) norm_bwd_kernel<1><<<grid, threads, 0, s>>>(a);
    else if (ch == 2) norm_bwd_kernel<2><<<grid, threads, 0, s>>>(a);
    else norm_bwd_kernel<4><<<grid, threads, 0, s>>>(a);
    MGQ_LAUNCH_CHECK();
  }
  norm_dw_kernel<<<(a.H + 31) / 32, 256, 0, s>>>(a.part, grid, a.H, beta, dw);
  MGQ_LAUNCH_CHECK();
  return MGQ_OK;
}
