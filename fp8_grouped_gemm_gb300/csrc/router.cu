// Top-k router: expert ids and probabilities from the router's logits, and the
// gradient of the logits from that of the probabilities.
//
// Scores of a row: s_e = softmax(l)_e or sigmoid(l_e). Both rise with the
// logit, so the k experts are the k largest logits (ties to the lower id).
//   p_j = scale s_j                    or, renormalised, scale s_j / S,  S = sum of the selected s
// Backward, d_j = dprobs_j, all sums over the selected experts:
//   softmax:               dl_e = s_e (G_e - sum_i s_i G_i),  G_e = scale d_j at the selected, 0 elsewhere
//   softmax, renormalised: dl_j = scale q_j (d_j - sum_i q_i d_i),  q = softmax over the selected
//   sigmoid:               dl_j = scale d_j s_j (1 - s_j)
//   sigmoid, renormalised: dl_j = scale / S (d_j - sum_i d_i s_i / S) s_j (1 - s_j)
//
// One warp takes one row and holds it in registers, lane l the V consecutive
// experts V l .. V l + V - 1, sorted. Each of the k rounds finds the largest
// ordered key among the lanes' heads with one integer warp reduction; the
// lowest lane that has it holds the lowest such id. No memory is touched
// between the load of the logits and the store of the k results.
#include "mgq_internal.h"
#include "device_common.cuh"
#include "ptx_sm100.cuh"

namespace mgq {
namespace {

constexpr uint32_t kFull = 0xFFFFFFFFu;
constexpr int kMaxTopK = 8;

// NaN ranks with the masked experts; -0 becomes +0
__device__ __forceinline__ float clean(float v) { return v != v ? -INFINITY : v + 0.0f; }
template <bool BF16>
__device__ __forceinline__ float load_logit(const void* p, int64_t i) {
  return clean(BF16 ? __uint_as_float(static_cast<uint32_t>(__ldg(static_cast<const uint16_t*>(p) + i)) << 16)
                    : __ldg(static_cast<const float*>(p) + i));
}
// unsigned key with the order of the floats; 0 is below every float's key
__device__ __forceinline__ uint32_t order_key(float v) {
  const uint32_t u = __float_as_uint(v);
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}
__device__ __forceinline__ float from_key(uint32_t k) {
  return __uint_as_float((k & 0x80000000u) ? (k & 0x7FFFFFFFu) : ~k);
}
__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(kFull, v, o);
  return v;
}
// sigmoid without overflow; 0 for -infinity
__device__ __forceinline__ float sigmoid_f32(float x) {
  const float e = expf(-fabsf(x));
  return x >= 0.0f ? 1.0f / (1.0f + e) : e / (1.0f + e);
}
// exp(x - m) of a softmax whose largest logit is m; a row with nothing but
// masked experts (m = -infinity) has no mass
__device__ __forceinline__ float softmax_term(float x, float m) { return m == -INFINITY ? 0.0f : expf(x - m); }

struct RouterArgs {
  const void* logits;
  int64_t T;
  int E, k, vec;
  float scale;
  int32_t* idx;
  float* probs;
  // backward
  const int32_t* sel;
  const float* dprobs;
  void* dlogits;
  int* err;
};

// the V logits of a row from expert e0 on; -infinity past the end (vec: whole
// aligned vectors)
template <int V, bool BF16>
__device__ __forceinline__ void load_row(const RouterArgs& a, int64_t r, int e0, float* v) {
  const int64_t at = r * a.E + e0;
  if (V >= 4 && a.vec) {
#pragma unroll
    for (int i = 0; i < V; i += 4) {
      if (e0 + i < a.E) {
        if (BF16) {
          const uint2 w = __ldg(reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(a.logits) + at + i));
          v[i] = bf16_lo(w.x), v[i + 1] = bf16_hi(w.x), v[i + 2] = bf16_lo(w.y), v[i + 3] = bf16_hi(w.y);
        } else {
          const float4 w = __ldg(reinterpret_cast<const float4*>(static_cast<const float*>(a.logits) + at + i));
          v[i] = w.x, v[i + 1] = w.y, v[i + 2] = w.z, v[i + 3] = w.w;
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) v[i + j] = clean(v[i + j]);
      } else {
#pragma unroll
        for (int j = 0; j < 4; ++j) v[i + j] = -INFINITY;
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i) v[i] = e0 + i < a.E ? load_logit<BF16>(a.logits, at + i) : -INFINITY;
  }
}

// sorts a lane's keys (largest first, equal keys in their order) with their
// experts e0 + i, a byte each: exchanges of neighbours only
template <int V>
__device__ __forceinline__ void sort_lane(uint32_t* key, int e0, uint32_t& at4) {
  uint32_t at[V];
#pragma unroll
  for (int i = 0; i < V; ++i) at[i] = e0 + i;
#pragma unroll
  for (int i = 1; i < V; ++i)
#pragma unroll
    for (int j = V - 1; j >= i; --j) {
      const bool swap = key[j] > key[j - 1];
      const uint32_t hi = max(key[j], key[j - 1]), lo = min(key[j], key[j - 1]);
      const uint32_t a0 = swap ? at[j] : at[j - 1], a1 = swap ? at[j - 1] : at[j];
      key[j - 1] = hi, key[j] = lo, at[j - 1] = a0, at[j] = a1;
    }
  at4 = 0;
#pragma unroll
  for (int i = 0; i < V; ++i) at4 |= at[i] << (8 * i);
}

// sum over the eight lanes of a row
__device__ __forceinline__ float sum8(float v) {
#pragma unroll
  for (int o = 4; o > 0; o >>= 1) v += __shfl_xor_sync(kFull, v, o);
  return v;
}

template <int V, bool BF16, bool SIGMOID, bool RENORM>
__global__ void __launch_bounds__(256) router_topk_kernel(RouterArgs a) {
  ptx::grid_wait();
  ptx::grid_launch();
  constexpr bool SORTED = V <= 4;     // longer runs: find the next best when the head is taken
  __shared__ uint16_t picked[8][kMaxTopK];
  uint16_t* pick = picked[threadIdx.x >> 5];
  const int lane = threadIdx.x & 31, e0 = lane * V;
  uint32_t below;                     // the lanes before this one
  asm("mov.u32 %0, %%lanemask_lt;" : "=r"(below));
  const int64_t nw = static_cast<int64_t>(gridDim.x) * (blockDim.x >> 5);
  for (int64_t r = blockIdx.x * static_cast<int64_t>(blockDim.x >> 5) + (threadIdx.x >> 5); r < a.T; r += nw) {
    float v[V];
    uint32_t key[V];
    load_row<V, BF16>(a, r, e0, v);
#pragma unroll
    for (int i = 0; i < V; ++i) key[i] = e0 + i < a.E ? order_key(v[i]) : 0u;
    uint32_t head = 0, at4 = 0;       // best key left; its expert in the low byte (or its place in the run)
    if (SORTED) {
      sort_lane<V>(key, e0, at4);
      head = key[0];
    } else {
#pragma unroll
      for (int i = 0; i < V; ++i)
        if (key[i] > head) head = key[i], at4 = i;
    }
    uint32_t k_sel = 0;   // lane j: the j-th selected key
    uint32_t top = 0;
    __syncwarp();         // the last row's picks are read
#pragma unroll
    for (int j = 0; j < kMaxTopK; ++j) {
      if (j >= a.k) break;
      const uint32_t m = __reduce_max_sync(kFull, head);
      const uint32_t have = __ballot_sync(kFull, head == m);
      if (lane == j) k_sel = m;
      if (j == 0) top = m;
      if (head == m && (have & below) == 0) {    // the owner takes it out
        pick[j] = static_cast<uint16_t>(SORTED ? at4 & 255u : e0 + at4);
        if (SORTED) {
#pragma unroll
          for (int i = 0; i + 1 < V; ++i) key[i] = key[i + 1];
          key[V - 1] = 0u;
          at4 >>= 8;
          head = key[0];
        } else {
          head = 0;
          const int taken = at4;
          at4 = 0;
#pragma unroll
          for (int i = 0; i < V; ++i) {
            if (i == taken) key[i] = 0;
            if (key[i] > head) head = key[i], at4 = i;
          }
        }
      }
    }
    __syncwarp();
    const bool on = lane < a.k;
    const float mx = from_key(top), l = from_key(k_sel);
    const float s = !on ? 0.0f : SIGMOID ? sigmoid_f32(l) : softmax_term(l, mx);
    float S = 1.0f;
    if (RENORM) {
      S = sum8(s);
    } else if (!SIGMOID) {
      S = 0.0f;
#pragma unroll
      for (int i = 0; i < V; ++i) S += softmax_term(v[i], mx);
      S = warp_sum(S);
    }
    if (on) {
      a.idx[r * a.k + lane] = pick[lane];
      a.probs[r * a.k + lane] = S == 0.0f ? 0.0f : a.scale * (s / S);
    }
  }
}

// A warp takes four rows at a time: eight lanes each work out the gradients of
// their row's selected logits, then all lanes write the four dense rows.
template <int V, bool BF16, bool SIGMOID, bool RENORM>
__global__ void __launch_bounds__(256) router_bwd_kernel(RouterArgs a) {
  ptx::grid_wait();
  ptx::grid_launch();
  // a dense row is put together in shared memory: zeros, the selected
  // experts' gradients by id, then V consecutive values a lane
  __shared__ __align__(16) float rows[8][32 * V];
  constexpr bool DENSE = !SIGMOID && !RENORM;      // every expert's score takes part
  const int lane = threadIdx.x & 31, e0 = lane * V, sub = lane & 7;
  float* row = rows[threadIdx.x >> 5];
#pragma unroll
  for (int i = 0; i < V; ++i) row[e0 + i] = 0.0f;
  const int64_t nw = static_cast<int64_t>(gridDim.x) * (blockDim.x >> 5);
  for (int64_t r4 = 4 * (blockIdx.x * static_cast<int64_t>(blockDim.x >> 5) + (threadIdx.x >> 5)); r4 < a.T; r4 += 4 * nw) {
    const int64_t r = r4 + (lane >> 3);
    int e = -1;
    float d = 0.0f;
    if (sub < a.k && r < a.T) {
      e = __ldg(a.sel + r * a.k + sub);
      d = __ldg(a.dprobs + r * a.k + sub);
      if (e < 0 || e >= a.E) {
        report(a.err, MGQ_ERR_DEVICE_INDEX);
        e = -1;
      }
    }
    const bool on = e >= 0;
    const float l = on ? load_logit<BF16>(a.logits, r * a.E + e) : -INFINITY;
    float g = 0.0f;         // the selected logit's own gradient (DENSE: dprobs times scale, for now)
    if (SIGMOID) {
      const float s = on ? sigmoid_f32(l) : 0.0f;
      if (RENORM) {
        const float S = sum8(s);
        const float q = S == 0.0f ? 0.0f : s / S;
        const float c = sum8(q > 0.0f ? d * q : 0.0f);
        g = q > 0.0f ? a.scale * (d - c) * q * sigmoid_f32(-l) : 0.0f;
      } else {
        g = s > 0.0f ? a.scale * d * s * sigmoid_f32(-l) : 0.0f;
      }
    } else if (RENORM) {
      float m = l;
#pragma unroll
      for (int o = 4; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(kFull, m, o));
      const float s = on ? softmax_term(l, m) : 0.0f;
      const float S = sum8(s);
      const float q = S == 0.0f ? 0.0f : s / S;
      const float c = sum8(q > 0.0f ? d * q : 0.0f);
      g = q > 0.0f ? a.scale * q * (d - c) : 0.0f;
    } else {
      g = a.scale * d;
    }
    const int nr = static_cast<int>(a.T - r4 < 4 ? a.T - r4 : 4);
    for (int t = 0; t < nr; ++t) {
      const int64_t rt = r4 + t;
      const bool own = on && (lane >> 3) == t;
      float v[V], top = 0.0f, back = 0.0f, gt = g;
      if (DENSE) {
        uint32_t km = 0;
        load_row<V, BF16>(a, rt, e0, v);
#pragma unroll
        for (int i = 0; i < V; ++i) km = max(km, order_key(v[i]));
        top = from_key(__reduce_max_sync(kFull, km));
        float all = 0.0f;
#pragma unroll
        for (int i = 0; i < V; ++i) all += softmax_term(v[i], top);
        all = warp_sum(all);
        const float inv = all == 0.0f ? 0.0f : 1.0f / all;
        const float s = own ? softmax_term(l, top) * inv : 0.0f;
        gt = s > 0.0f ? g * s : 0.0f;
        back = warp_sum(gt) * inv;
      }
      if (own) atomicAdd(row + e, gt);    // (ids of a row are distinct: one addition each)
      __syncwarp();
      float o[V];
#pragma unroll
      for (int i = 0; i < V; ++i) {
        o[i] = row[e0 + i];
        row[e0 + i] = 0.0f;
        if (DENSE) o[i] -= softmax_term(v[i], top) * back;
      }
      __syncwarp();
      const int64_t at = rt * a.E + e0;
      if (V >= 4 && a.vec) {
#pragma unroll
        for (int i = 0; i < V; i += 4) {
          if (e0 + i >= a.E) continue;
          if (BF16)
            *reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.dlogits) + at + i) =
                make_uint2(pack_bf16x2(o[i], o[i + 1]), pack_bf16x2(o[i + 2], o[i + 3]));
          else
            *reinterpret_cast<float4*>(static_cast<float*>(a.dlogits) + at + i) =
                make_float4(o[i], o[i + 1], o[i + 2], o[i + 3]);
        }
      } else {
#pragma unroll
        for (int i = 0; i < V; ++i) {
          if (e0 + i >= a.E) continue;
          if (BF16) static_cast<__nv_bfloat16*>(a.dlogits)[at + i] = __float2bfloat16_rn(o[i]);
          else static_cast<float*>(a.dlogits)[at + i] = o[i];
        }
      }
    }
  }
}

template <int V, bool BF16>
bool launch_mode(const RouterArgs& a, bool bwd, bool sigmoid, bool renorm, int grid, cudaStream_t s) {
  void (*kern)(RouterArgs);
  if (bwd)
    kern = sigmoid ? (renorm ? router_bwd_kernel<V, BF16, true, true> : router_bwd_kernel<V, BF16, true, false>)
                   : (renorm ? router_bwd_kernel<V, BF16, false, true> : router_bwd_kernel<V, BF16, false, false>);
  else
    kern = sigmoid ? (renorm ? router_topk_kernel<V, BF16, true, true> : router_topk_kernel<V, BF16, true, false>)
                   : (renorm ? router_topk_kernel<V, BF16, false, true> : router_topk_kernel<V, BF16, false, false>);
  return launch_after(kern, dim3(grid), 256, 0, 1, s, a);
}

template <bool BF16>
int launch_router(RouterArgs a, bool bwd, bool sigmoid, bool renorm, cudaStream_t s) {
  // vectors of four logits: rows of a multiple of four, aligned bases
  const uintptr_t size = BF16 ? 8 : 16;
  a.vec = a.E % 4 == 0 && ((reinterpret_cast<uintptr_t>(a.logits) | reinterpret_cast<uintptr_t>(a.dlogits)) & (size - 1)) == 0;
  const int64_t per = bwd ? 32 : 8;      // rows of a CTA at a time
  const int64_t ctas = (a.T + per - 1) / per, most = static_cast<int64_t>(num_sms()) * 8;
  const int grid = static_cast<int>(ctas < most ? ctas : most);
  auto go = a.E <= 32 ? launch_mode<1, BF16> : a.E <= 64 ? launch_mode<2, BF16> : a.E <= 128 ? launch_mode<4, BF16> :
            a.E <= 256 ? launch_mode<8, BF16> : a.E <= 512 ? launch_mode<16, BF16> : launch_mode<32, BF16>;
  return go(a, bwd, sigmoid, renorm, grid, s) ? MGQ_OK : MGQ_ERR_CUDA;
}

int check_router(const void* logits, int dtype, int64_t T, int E, int k, int score, int renorm) {
  MGQ_CHECK_ARG(dtype == MGQ_OUT_BF16 || dtype == MGQ_OUT_F32);
  MGQ_CHECK_ARG(score == MGQ_SCORE_SOFTMAX || score == MGQ_SCORE_SIGMOID);
  MGQ_CHECK_ARG(renorm == 0 || renorm == 1);
  MGQ_CHECK_ARG(T >= 0 && T <= (int64_t(1) << 40) && E >= 1 && E <= 1024 && k >= 1 && k <= kMaxTopK && k <= E);
  MGQ_CHECK_ARG(T == 0 || logits);
  const uintptr_t size = dtype == MGQ_OUT_BF16 ? 2 : 4;
  MGQ_CHECK_ARG((reinterpret_cast<uintptr_t>(logits) & (size - 1)) == 0);
  return MGQ_OK;
}

}  // namespace
}  // namespace mgq

using namespace mgq;

extern "C" int mgq_router_topk(const void* logits, int dtype, int64_t T, int E, int k, int score, int renorm,
                               float scale, int32_t* topk_idx, float* probs, void* stream) {
  const int rc = check_router(logits, dtype, T, E, k, score, renorm);
  if (rc != MGQ_OK) return rc;
  if (T == 0) return MGQ_OK;
  MGQ_CHECK_ARG(topk_idx && probs);
  RouterArgs a{};
  a.logits = logits;
  a.T = T;
  a.E = E;
  a.k = k;
  a.scale = scale;
  a.idx = topk_idx;
  a.probs = probs;
  const bool sig = score == MGQ_SCORE_SIGMOID;
  return dtype == MGQ_OUT_BF16 ? launch_router<true>(a, false, sig, renorm != 0, as_stream(stream))
                               : launch_router<false>(a, false, sig, renorm != 0, as_stream(stream));
}

extern "C" int mgq_router_topk_bwd(const void* logits, int dtype, const int32_t* topk_idx, const float* dprobs,
                                   int64_t T, int E, int k, int score, int renorm, float scale, void* dlogits,
                                   void* stream) {
  const int rc = check_router(logits, dtype, T, E, k, score, renorm);
  if (rc != MGQ_OK) return rc;
  if (T == 0) return MGQ_OK;
  MGQ_CHECK_ARG(topk_idx && dprobs && dlogits);
  MGQ_CHECK_ARG((reinterpret_cast<uintptr_t>(dlogits) & (dtype == MGQ_OUT_BF16 ? 1 : 3)) == 0);
  RouterArgs a{};
  a.logits = logits;
  a.T = T;
  a.E = E;
  a.k = k;
  a.scale = scale;
  a.sel = topk_idx;
  a.dprobs = dprobs;
  a.dlogits = dlogits;
  a.err = error_word();
  const bool sig = score == MGQ_SCORE_SIGMOID;
  return dtype == MGQ_OUT_BF16 ? launch_router<true>(a, true, sig, renorm != 0, as_stream(stream))
                               : launch_router<false>(a, true, sig, renorm != 0, as_stream(stream));
}
