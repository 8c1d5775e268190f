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
// Few rows: one warp takes one row and holds it in registers, lane l the V
// consecutive experts V l .. V l + V - 1, sorted. Each of the k rounds finds the
// largest ordered key among the lanes' heads with one integer warp reduction;
// the lowest lane that has it holds the lowest such id. 16 rows of 128, top 8:
// 1.5 us, most of it the launch and one trip to memory.
#include "mgq_internal.h"
#include "device_common.cuh"
#include "ptx_sm100.cuh"

namespace mgq {
namespace {

constexpr uint32_t kFull = 0xFFFFFFFFu;
constexpr int kMaxTopK = 8;

// NaN ranks with the masked experts; -0 becomes +0
__device__ __forceinline__ float clean(float v) { return fmaxf(v, -INFINITY) + 0.0f; }
// (Plain loads, not those of the read-only path: the launch before may still be
// writing when these kernels start.)
template <bool BF16>
__device__ __forceinline__ float load_logit(const void* p, int64_t i) {
  return clean(BF16 ? __uint_as_float(static_cast<uint32_t>(static_cast<const uint16_t*>(p)[i]) << 16)
                    : static_cast<const float*>(p)[i]);
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
  int E, k, vec, sigmoid, renorm;
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
          const uint2 w = *reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(a.logits) + at + i);
          v[i] = bf16_lo(w.x), v[i + 1] = bf16_hi(w.x), v[i + 2] = bf16_lo(w.y), v[i + 3] = bf16_hi(w.y);
        } else {
          const float4 w = *reinterpret_cast<const float4*>(static_cast<const float*>(a.logits) + at + i);
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

// ---- many rows: G lanes a row -------------------------------------------------
//
// A round of the kernel above costs a warp reduction for one row (32 cycles of
// a scheduler). Here G lanes hold a row, V consecutive experts each, and a warp
// works on 32 / G rows: the keys alone are sorted, by networks of minima and
// maxima, and the best eight of a lane kept; a round is log2 G exchanges for
// all the rows. Which expert a key stands for is found at the end, by thread j
// of a row for its pick j: it reads the run of the lane that had it once more
// and takes the first equal logit, the t-th if the lane gave that
// value t times before. Sums in the other kernel's order: the same bits.
//
// Bound by the rounds' dependent exchanges at the warps that 48 registers a
// thread allow (fewer registers spill: six CTAs an SM 8.9 us, seven 11.3); issue
// and compare pipe are half busy, 148 warp instructions a row of 128. 32768 rows
// of 128, top 8: 8.2 us, 18.9 MB at 2.3 TB/s.

__device__ __forceinline__ void order2(float& hi, float& lo) {
  const float a = fmaxf(hi, lo), b = fminf(hi, lo);
  hi = a, lo = b;
}
// Batcher's odd-even merge sort of eight (19 exchanges) or of four, descending
template <int N>
__device__ __forceinline__ void sort_keys(float* k) {
#pragma unroll
  for (int p = 1; p < N; p <<= 1)
#pragma unroll
    for (int q = p; q > 0; q >>= 1)
#pragma unroll
      for (int j = q % p; j + q < N; j += 2 * q)
#pragma unroll
        for (int i = 0; i < q; ++i)
          if (i + j + q < N && (i + j) / (2 * p) == (i + j + q) / (2 * p)) order2(k[i + j], k[i + j + q]);
}

// a row's logits as G lanes read them together: vectors of four (or single
// ones) in turn; -infinity past the end
template <int G, int V, bool BF16>
__device__ __forceinline__ void load_strided(const RouterArgs& a, int64_t r, int sub, float* v) {
  if (a.vec) {
#pragma unroll
    for (int i = 0; i < V; i += 4) load_row<4, BF16>(a, r, 4 * sub + G * i, v + i);
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i) load_row<1, BF16>(a, r, sub + G * i, v + i);
  }
}
template <int V>
__device__ __forceinline__ void load_run(const float* p, float* v) {
#pragma unroll
  for (int i = 0; i < V; i += 4) {
    const float4 w = *reinterpret_cast<const float4*>(p + i);
    v[i] = w.x, v[i + 1] = w.y, v[i + 2] = w.z, v[i + 3] = w.w;
  }
}

template <int G, int V, bool BF16>
__global__ void __launch_bounds__(256) router_topk_rows_kernel(RouterArgs a) {
  ptx::grid_wait();
  ptx::grid_launch();
  constexpr int KEEP = V < kMaxTopK ? V : kMaxTopK, ROWS = 32 / G;
  // the rows' logits, a run of V every LD floats: eight runs lie in different banks
  constexpr int LD = V == 4 ? 4 : V + 4;
  __shared__ __align__(16) float logits[8][32 * LD];
  __shared__ float2 picked[8][ROWS][kMaxTopK];    // a pick: the logit, the lane of its row that had it
  const int lane = threadIdx.x & 31, sub = lane % G, base = lane - sub;
  float2* pick = picked[threadIdx.x >> 5][lane / G];
  float* row = logits[threadIdx.x >> 5] + base * LD;
  const uint32_t before = ((1u << sub) - 1u) << base;     // the row's lanes before this one
  const int64_t nw = static_cast<int64_t>(gridDim.x) * (blockDim.x >> 5);
  for (int64_t r0 = ROWS * (blockIdx.x * static_cast<int64_t>(blockDim.x >> 5) + (threadIdx.x >> 5)); r0 < a.T;
       r0 += ROWS * nw) {
    const int64_t r = r0 + lane / G;
    const bool live = r < a.T;
    float v[V];
    __syncwarp();         // the last rows are read
    load_strided<G, V, BF16>(a, live ? r : r0, sub, v);
    if (a.vec) {
#pragma unroll
      for (int i = 0; i < V; i += 4) {
        const int e = 4 * sub + G * i;
        *reinterpret_cast<float4*>(row + e / V * LD + e % V) = make_float4(v[i], v[i + 1], v[i + 2], v[i + 3]);
      }
    } else {
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const int e = sub + G * i;
        row[e / V * LD + e % V] = v[i];
      }
    }
    __syncwarp();
    load_run<V>(row + sub * LD, v);
    // A taken key becomes NaN, which loses to every number. Places past the end
    // are -infinity: a row's own experts come before them, and there are k.
    float key[V];
#pragma unroll
    for (int i = 0; i < V; ++i) key[i] = v[i];
    if constexpr (V <= 8) {
      sort_keys<V>(key);
    } else {
      sort_keys<8>(key);
      sort_keys<8>(key + 8);
#pragma unroll
      for (int i = 0; i < 8; ++i) key[i] = fmaxf(key[i], key[15 - i]);     // the best eight, rising and falling
#pragma unroll
      for (int q = 4; q > 0; q >>= 1)
#pragma unroll
        for (int i = 0; i < 8; ++i)
          if (!(i & q)) order2(key[i], key[i + q]);
    }
    float mx = 0.0f;
#pragma unroll
    for (int j = 0; j < kMaxTopK; ++j) {
      if (j >= a.k) break;
      float m = key[0];
#pragma unroll
      for (int o = 1; o < G; o <<= 1) m = fmaxf(m, __shfl_xor_sync(kFull, m, o));
      const bool has = key[0] == m;
      const uint32_t have = __ballot_sync(kFull, has);
      if (j == 0) mx = m;
      if (has && (have & before) == 0) {
        pick[j] = make_float2(m, __int_as_float(sub));
#pragma unroll
        for (int i = 0; i + 1 < KEEP; ++i) key[i] = key[i + 1];
        key[KEEP - 1] = __uint_as_float(0x7FC00000u);
      }
    }
    __syncwarp();
    const bool on = sub < a.k;
    const float2 mine = on ? pick[sub] : make_float2(0.0f, 0.0f);
    const float l = mine.x;
    const int w = __float_as_int(mine.y);
    float s = 0.0f, S = 1.0f;
    if (on) s = a.sigmoid ? sigmoid_f32(l) : softmax_term(l, mx);
    if (a.renorm) {
      S = sum8(s);
    } else if (!a.sigmoid) {
      constexpr int P = 32 / G;       // the runs of this lane that a lane each has in the kernel above
      float part[P];
#pragma unroll
      for (int t = 0; t < P; ++t) {
        part[t] = 0.0f;
#pragma unroll
        for (int i = 0; i < V / P; ++i) part[t] += softmax_term(v[t * (V / P) + i], mx);
#pragma unroll
        for (int o = G / 2; o > 0; o >>= 1) part[t] += __shfl_xor_sync(kFull, part[t], o);
      }
#pragma unroll
      for (int n = P / 2; n > 0; n >>= 1)
#pragma unroll
        for (int t = 0; t < n; ++t) part[t] += part[t + n];
      S = part[0];
    }
    load_run<V>(row + w * LD, v);
    uint32_t same = 0;
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (v[i] == l) same |= 1u << i;
    if (__any_sync(kFull, on && (same & (same - 1)) != 0)) {
      int t = 0;
      for (int j = 0; j + 1 < a.k; ++j) {
        const float lj = __shfl_sync(kFull, l, base + j);
        const int wj = __shfl_sync(kFull, w, base + j);
        t += j < sub && lj == l && wj == w;
      }
      for (; t > 0; --t) same &= same - 1;
    }
    if (on && live) {
      a.idx[r * a.k + sub] = w * V + __ffs(same) - 1;
      a.probs[r * a.k + sub] = S == 0.0f ? 0.0f : a.scale * (s / S);
    }
  }
}

// ---- backward ------------------------------------------------------------------

// G lanes a row, 32 / G rows a warp: lane j < k of a row works out the gradient
// of its j-th selected logit; they meet in shared memory as a dense row, which
// the G lanes write out in vectors of four. DENSE (softmax over all experts,
// not renormalised): every expert's score takes part, read the same way. No
// warp has more than its 32 / G rows to do before T fills the GPU; what is left
// is three trips to memory, one after the other, and the write. 16 rows of 128:
// 2.0 us (DENSE 2.8); 32768 rows, float32: 7.2 us at 2.6 TB/s (DENSE 10.3 us at
// 3.5 TB/s); 32768 rows of 1024: 31 us at 4.4 TB/s.
template <int G, int V, bool BF16, bool DENSE>
__global__ void __launch_bounds__(256, DENSE ? 4 : 6) router_bwd_kernel(RouterArgs a) {
  ptx::grid_wait();
  ptx::grid_launch();
  constexpr int ROWS = 32 / G;
  __shared__ __align__(16) float rows[8][32 * V];
  const int lane = threadIdx.x & 31, sub = lane % G;
  float* row = rows[threadIdx.x >> 5] + lane / G * (G * V);
#pragma unroll
  for (int i = 0; i < V; ++i) row[sub + G * i] = 0.0f;
  __syncwarp();
  const int64_t nw = static_cast<int64_t>(gridDim.x) * (blockDim.x >> 5);
  for (int64_t r0 = ROWS * (blockIdx.x * static_cast<int64_t>(blockDim.x >> 5) + (threadIdx.x >> 5)); r0 < a.T;
       r0 += ROWS * nw) {
    const int64_t r = r0 + lane / G;
    const bool live = r < a.T;
    float v[DENSE ? V : 1];
    if constexpr (DENSE) load_strided<G, V, BF16>(a, live ? r : r0, sub, v);
    int e = -1;
    float d = 0.0f;
    if (sub < a.k && live) {
      e = a.sel[r * a.k + sub];
      d = a.dprobs[r * a.k + sub];
      if (e < 0 || e >= a.E) {
        report(a.err, MGQ_ERR_DEVICE_INDEX);
        e = -1;
      }
    }
    const bool on = e >= 0;
    // loaded by every lane: a branch here costs the row's lanes 0.9 us
    const float at_e = load_logit<BF16>(a.logits, (live ? r : r0) * a.E + (on ? e : 0));
    const float l = on ? at_e : -INFINITY;
    float g = 0.0f, back = 0.0f;
    if constexpr (DENSE) {
      float top = v[0];
#pragma unroll
      for (int i = 1; i < V; ++i) top = fmaxf(top, v[i]);
#pragma unroll
      for (int o = G / 2; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(kFull, top, o));
      float all = 0.0f;
#pragma unroll
      for (int i = 0; i < V; ++i) all += v[i] = softmax_term(v[i], top);
#pragma unroll
      for (int o = G / 2; o > 0; o >>= 1) all += __shfl_xor_sync(kFull, all, o);
      const float inv = all == 0.0f ? 0.0f : 1.0f / all;
      const float s = on ? softmax_term(l, top) * inv : 0.0f;
      g = s > 0.0f ? a.scale * d * s : 0.0f;
      back = g;
#pragma unroll
      for (int o = G / 2; o > 0; o >>= 1) back += __shfl_xor_sync(kFull, back, o);
      back *= inv;
    } else if (a.sigmoid) {
      const float s = on ? sigmoid_f32(l) : 0.0f;
      if (a.renorm) {
        const float S = sum8(s);
        const float q = s * (1.0f / (S == 0.0f ? 1.0f : S));
        const float c = sum8(q > 0.0f ? d * q : 0.0f);
        g = q > 0.0f ? a.scale * (d - c) * q * sigmoid_f32(-l) : 0.0f;
      } else {
        g = s > 0.0f ? a.scale * d * s * sigmoid_f32(-l) : 0.0f;
      }
    } else {
      float m = l;
#pragma unroll
      for (int o = 4; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(kFull, m, o));
      const float s = on ? softmax_term(l, m) : 0.0f;
      const float S = sum8(s);
      const float q = s * (1.0f / (S == 0.0f ? 1.0f : S));
      const float c = sum8(q > 0.0f ? d * q : 0.0f);
      g = q > 0.0f ? a.scale * q * (d - c) : 0.0f;
    }
    if (on) atomicAdd(row + e, g);    // (ids of a row are distinct: one addition each)
    __syncwarp();
    const int64_t at = r * a.E;
    if (a.vec) {
#pragma unroll
      for (int i = 0; i < V; i += 4) {
        const int c = 4 * sub + G * i;
        float4 o = *reinterpret_cast<float4*>(row + c);
        *reinterpret_cast<float4*>(row + c) = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        if constexpr (DENSE)
          o.x -= v[i] * back, o.y -= v[i + 1] * back, o.z -= v[i + 2] * back, o.w -= v[i + 3] * back;
        if (live && c < a.E) {
          if (BF16)
            *reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.dlogits) + at + c) =
                make_uint2(pack_bf16x2(o.x, o.y), pack_bf16x2(o.z, o.w));
          else
            *reinterpret_cast<float4*>(static_cast<float*>(a.dlogits) + at + c) = o;
        }
      }
    } else {
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const int c = sub + G * i;
        float o = row[c];
        row[c] = 0.0f;
        if constexpr (DENSE) o -= v[i] * back;
        if (live && c < a.E) {
          if (BF16) static_cast<__nv_bfloat16*>(a.dlogits)[at + c] = __float2bfloat16_rn(o);
          else static_cast<float*>(a.dlogits)[at + c] = o;
        }
      }
    }
    __syncwarp();
  }
}

bool launch_grid(void (*kern)(RouterArgs), int64_t rows, const RouterArgs& a, cudaStream_t s) {
  const int64_t ctas = (a.T + rows - 1) / rows, most = static_cast<int64_t>(num_sms()) * 8;
  return launch_after(kern, dim3(static_cast<unsigned>(ctas < most ? ctas : most)), 256, 0, 1, s, a);
}

template <int V, bool BF16>
bool launch_topk(const RouterArgs& a, cudaStream_t s) {
  return launch_grid(a.sigmoid ? (a.renorm ? router_topk_kernel<V, BF16, true, true> : router_topk_kernel<V, BF16, true, false>)
                               : (a.renorm ? router_topk_kernel<V, BF16, false, true> : router_topk_kernel<V, BF16, false, false>),
                     8, a, s);
}
template <int G, int V, bool BF16>
bool launch_topk_rows(const RouterArgs& a, cudaStream_t s) {
  return launch_grid(router_topk_rows_kernel<G, V, BF16>, 8 * (32 / G), a, s);
}
template <int G, int V, bool BF16>
bool launch_bwd(const RouterArgs& a, cudaStream_t s) {
  return launch_grid(!a.sigmoid && !a.renorm ? router_bwd_kernel<G, V, BF16, true> : router_bwd_kernel<G, V, BF16, false>,
                     8 * (32 / G), a, s);
}

// Which kernel takes the forward pass: G lanes a row once that gives every SM
// eight warps. Measured on 152 SMs (38912 lanes), float32, top 8, a warp a row / G lanes:
//   E 128  T  4096  2.88 /  2.82 us    8192  4.60 / 3.43    32768  12.8 /  8.2
//   E 256  T  1216  2.69 /  2.97 us    2432  3.50 / 3.00    32768  26.3 / 14.8
//   E 512  T   608  3.45 /  3.01 us    2432  5.10 / 3.75    32768  46.3 / 27.8
bool many_rows(int64_t T, int E) {
  const int G = E <= 128 ? 8 : E <= 256 ? 16 : 32;
  return E <= 512 && T * G >= static_cast<int64_t>(num_sms()) * 8 * 32;
}

template <bool BF16>
int launch_router(RouterArgs a, bool bwd, bool sigmoid, bool renorm, cudaStream_t s) {
  // vectors of four logits: rows of a multiple of four, aligned bases
  const uintptr_t size = BF16 ? 8 : 16;
  a.vec = a.E % 4 == 0 && ((reinterpret_cast<uintptr_t>(a.logits) | reinterpret_cast<uintptr_t>(a.dlogits)) & (size - 1)) == 0;
  a.sigmoid = sigmoid, a.renorm = renorm;
  const int E = a.E;
  auto go = bwd ? (E <= 32    ? launch_bwd<8, 4, BF16>
                   : E <= 64  ? launch_bwd<8, 8, BF16>
                   : E <= 128 ? launch_bwd<8, 16, BF16>
                   : E <= 256 ? launch_bwd<16, 16, BF16>
                   : E <= 512 ? launch_bwd<32, 16, BF16>
                              : launch_bwd<32, 32, BF16>)
            : many_rows(a.T, E) ? (E <= 32    ? launch_topk_rows<8, 4, BF16>
                                   : E <= 64  ? launch_topk_rows<8, 8, BF16>
                                   : E <= 128 ? launch_topk_rows<8, 16, BF16>
                                   : E <= 256 ? launch_topk_rows<16, 16, BF16>
                                              : launch_topk_rows<32, 16, BF16>)
                                : (E <= 32    ? launch_topk<1, BF16>
                                   : E <= 64  ? launch_topk<2, BF16>
                                   : E <= 128 ? launch_topk<4, BF16>
                                   : E <= 256 ? launch_topk<8, BF16>
                                   : E <= 512 ? launch_topk<16, BF16>
                                              : launch_topk<32, BF16>);
  return go(a, s) ? MGQ_OK : MGQ_ERR_CUDA;
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
