// The whole routed-expert layer for a few tokens (decode): T of 1 to 128.
//
//   out[t] = sum_j probs[t, j] W2_e Q(silu(g) u),   [g | u] = W1_e Q(x_t),   e = topk_idx[t, j]
//
// With so few rows the layer is bound by reading the weights of the experts
// that were picked, once. The grouped GEMMs put tokens on the 128 rows of the
// tensor-core tile, so a group of one token costs 128 padded rows; here the
// operands change places: 128 rows of a weight are the tile's M and the
// expert's tokens (at most 64 a tile, in steps of 16) its N. The weights' codes
// and block scales go from memory to shared memory by TMA and into the MMA as
// they are, and nothing is padded in memory.
//
// Four launches, each started while the one before drains (programmatic
// dependent launch):
//   few_prep_kernel   rows of the routed tokens in expert order, quantised
//   few_gemm_kernel   gate and up rows of W1, SwiGLU, h quantised
//   few_gemm_kernel   W2, rows of y in float32
//   few_combine_kernel  out[t] = sum_j probs y
// A GEMM's work is a line of units, one per (tile, 128 bytes of contraction),
// 32 KB of weight each; every CTA takes an equal stretch of it, whatever the
// number of tiles. A tile that two or more CTAs share is joined by the last of
// them to finish: the others leave float32 partial sums, which it adds in the
// order of the CTAs, so the result does not depend on who came last. Nobody
// waits for another CTA.
//
// Measured (all four launches; weights / time): one token, 2 experts of (H 4096,
// F 14336), MXFP8, 363 MB in 65 us, 5.6 TB/s; 16 tokens, all 8 of them, per
// tensor, 1.41 GB in 214 us, 6.6 TB/s; 64 tokens, 126 of 128 experts of (2048,
// 768), NVFP4, 335 MB in 65 us, 5.2 TB/s; 33 tokens, 14, 14 and 16 of 16 experts of
// (5120, 8192) in turn, 1x128, 1.85 GB in 277 us, 6.7 TB/s. What is not the weights' read is
// about 12 us: four starts, the last tiles' epilogues and joins. Small experts
// with many tokens are bound by the epilogue: 101 tokens on 4 of (512, 768), 14 us
// per tensor, 21 us NVFP4.
#include "moe_few.h"
#include "ptx_sm100.cuh"
#include "rowquant.cuh"

namespace mgq {
namespace {

constexpr int kMaxT = 128, kMaxK = 8, kMaxE = 1024;
constexpr int kTok = 64;                  // tokens of one tile (tensor-memory columns of one half)
constexpr int kEpiWarps = 8;              // two groups of four: one thread a weight row each, half of the tokens
constexpr int kThreads = 64 + 32 * kEpiWarps;   // warp 0 TMA, warp 1 MMA, the others the epilogue
constexpr uint32_t kATile = 128 * 128;    // bytes of 128 weight rows of one stage
constexpr int kMaxStages = 6;
constexpr int kBars = 26;                 // 8-byte words of the barriers and flags

__host__ __device__ constexpr uint32_t sf_chunks(int kind) { return kind == kMX ? 1 : kind == kNV ? 4 : 0; }
// scale bytes of one stage: two weight halves and the tokens (BLK: 64 float32 of the tokens)
__host__ __device__ constexpr uint32_t sf_bytes(int kind) { return kind == kBLK ? 256u : 3 * 512 * sf_chunks(kind); }

using ptx::grid_launch;
using ptx::grid_wait;
// true in one lane of the (converged) warp. Unlike a test of the lane index it
// tells the compiler that one thread is left, so that the operands of TMA and
// MMA instructions are kept in uniform registers.
__device__ __forceinline__ bool elect_one() {
  uint32_t r;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xFFFFFFFF;\n\tselp.b32 %0, 1, 0, p;\n\t}" : "=r"(r));
  return r != 0;
}
// the epilogue warps
__device__ __forceinline__ void epi_sync() { asm volatile("bar.sync 1, %0;" ::"n"(32 * kEpiWarps) : "memory"); }
// one group of them
__device__ __forceinline__ void group_sync(int grp) { asm volatile("bar.sync %0, 128;" ::"r"(2 + grp) : "memory"); }
// the first barrier, true if `ok` is true in all the warps (a wait that ran out
// in one of them must not leave the others at a barrier that it never reaches)
__device__ __forceinline__ bool epi_all(bool ok) {
  uint32_t r;
  asm volatile("{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\tbarrier.cta.red.and.pred q, 1, %2, p;\n\t"
               "selp.u32 %0, 1, 0, q;\n\t}"
               : "=r"(r)
               : "r"(static_cast<uint32_t>(ok)), "n"(32 * kEpiWarps)
               : "memory");
  return r != 0;
}

__device__ __forceinline__ uint32_t cvt_e2m1x2(float lo, float hi) {
  uint32_t r;
  asm("{\n\t.reg .b8 b;\n\tcvt.rn.satfinite.e2m1x2.f32 b, %2, %1;\n\tmov.b32 %0, {b, b, b, b};\n\t}"
      : "=r"(r)
      : "f"(lo), "f"(hi));
  return r & 0xFFu;
}

// ---------------------------------------------------------------------------
// Routed rows. Row order: by expert, then by entry i = t k + j. Tokens of an
// expert fall into blocks of 64; block b of an expert whose rows start at s
// keeps its scales in slot s / 64 + b + e, unique because a later block starts
// at least one row further on and a later expert has a larger e.

struct PrepArgs {
  const uint16_t* x;
  const int32_t* idx;
  int R, k, E;
  int H;
  uint8_t* xq;
  uint8_t* xs;
  const float* x_scale;
  int32_t* row_of;     // [R]
  int32_t* cnt;        // arrival counters to clear
  int ncnt;
  int* err;
};

template <int KIND>
__global__ void __launch_bounds__(128) few_prep_kernel(PrepArgs a) {
  // The next launch reads the ids and the weights before it waits for this one:
  // they must be there. From here on they and what else the layer was given can
  // be read through the read-only path; in this kernel, which may start while
  // they are written, loads are plain.
  grid_wait();
  grid_launch();
  const uint32_t lane = threadIdx.x & 31;
  if (blockIdx.x == 0)
    for (int i = threadIdx.x; i < a.ncnt; i += 128) a.cnt[i] = 0;
  const int nchunk = (a.H + 1023) / 1024;
  const int wid = blockIdx.x * 4 + (threadIdx.x >> 5);
  const int i = wid / nchunk, ck = wid - i * nchunk;
  if (i >= a.R) return;
  const int e = a.idx[i];
  if (e < 0 || e >= a.E) {
    if (ck == 0 && lane == 0) {
      a.row_of[i] = -1;
      report(a.err, MGQ_ERR_DEVICE_INDEX);
    }
    return;
  }
  int before = 0, same = 0;     // entries of lower experts; earlier entries of this one
  for (int q = lane; q < a.R; q += 32) {
    const int f = a.idx[q];
    before += f >= 0 && f < e;
    same += f == e && q < i;
  }
  before = __reduce_add_sync(0xFFFFFFFFu, before);
  same = __reduce_add_sync(0xFFFFFFFFu, same);
  const int row = before + same;
  if (ck == 0 && lane == 0) a.row_of[i] = row;
  const int64_t slot = before / kTok + same / kTok + e;
  const uint32_t n = same % kTok;
  const int c = ck * 1024 + lane * 32;
  float v[32];
  const bool in = c < a.H;
  if (in) {
    const uint4* p = reinterpret_cast<const uint4*>(a.x + static_cast<int64_t>(i / a.k) * a.H + c);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const uint4 w = p[j];
      v[8 * j] = bf16_lo(w.x), v[8 * j + 1] = bf16_hi(w.x), v[8 * j + 2] = bf16_lo(w.y), v[8 * j + 3] = bf16_hi(w.y);
      v[8 * j + 4] = bf16_lo(w.z), v[8 * j + 5] = bf16_hi(w.z), v[8 * j + 6] = bf16_lo(w.w), v[8 * j + 7] = bf16_hi(w.w);
    }
  } else {
#pragma unroll
    for (int j = 0; j < 32; ++j) v[j] = 0.0f;
  }
  const uint32_t in_chunk = (n & 31) * 16 + (n >> 5) * 4;    // the token's place in a 512-byte scale chunk
  if (KIND == kNV) {
    Block32nv b;
    quantize32_nv(v, *a.x_scale, b);
    if (in) {
      *reinterpret_cast<uint4*>(a.xq + static_cast<int64_t>(row) * (a.H / 2) + c / 2) =
          make_uint4(b.cw[0], b.cw[1], b.cw[2], b.cw[3]);
      if ((lane & 1) == 0) *reinterpret_cast<uint32_t*>(a.xs + (slot * (a.H / 64) + c / 64) * 512 + in_chunk) = b.s4;
    }
  } else {
    constexpr int SC = KIND == kMX ? MGQ_MX32_E8M0 : MGQ_TENSOR_F32;
    Block32 b;
    if (KIND == kBLK) {
      uint32_t m = absmax_bits_f32(v, 32);
      m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, 1));
      m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, 2));
      const float mult = blk_scale_few(m);
      b.sinv = __fdiv_rn(1.0f, mult);
#pragma unroll
      for (int j = 0; j < 8; ++j)
        b.cw[j] = cvt_fp8x4_mul<MGQ_E4M3>(v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3], mult);
    } else {
      quantize32<SC, MGQ_E4M3>(v, absmax_bits_f32(v, 32), KIND == kTEN ? *a.x_scale : 1.0f, true, b);
    }
    if (in) {
      uint4* dst = reinterpret_cast<uint4*>(a.xq + static_cast<int64_t>(row) * a.H + c);
      dst[0] = make_uint4(b.cw[0], b.cw[1], b.cw[2], b.cw[3]);
      dst[1] = make_uint4(b.cw[4], b.cw[5], b.cw[6], b.cw[7]);
      if ((lane & 3) == 0) {
        if (KIND == kMX) *reinterpret_cast<uint32_t*>(a.xs + (slot * (a.H / 128) + c / 128) * 512 + in_chunk) = b.s4;
        if (KIND == kBLK) reinterpret_cast<float*>(a.xs)[(slot * (a.H / 128) + c / 128) * kTok + n] = b.sinv;
      }
    }
  }
}

// ---------------------------------------------------------------------------
// The two GEMMs. PHASE 1: 128 gate rows and the matching 128 up rows of W1 are
// the two halves of a tile; PHASE 2: 256 consecutive rows of W2 (the second
// half may be missing at the end).

struct FewArgs {
  const int32_t* idx;
  int R, E;
  int64_t rows_e;        // weight rows of an expert
  int mt, kb;            // tiles along M, stages along the contraction
  int half2;             // rows from the first half to the second
  int mstep;             // rows from one tile to the next
  int rows_end;          // phase 2: rows of an expert that exist
  int kblk;              // BLK: 128-blocks of the contraction
  const uint8_t* sfa;    // weight block scales (MX, NV), chunks of 512 bytes
  int64_t sfa_kb4;       // chunks per 128 rows
  const float* sw;       // TEN: s per expert; NV: s_g per expert; BLK: scale_inv
  const uint8_t* sfb;    // token scales, by slot
  const float* sx;       // TEN, NV: scale of the tokens' operand
  float* part;           // [2 grid][nmax * 256]
  int32_t* cnt;          // [grid]
  int nmax;              // tokens a place of `part` can hold (multiple of 16, at most 64)
  int list;              // experts that can be active at once
  uint32_t stage_mem;    // shared memory for the stages
  uint32_t idesc0;       // instruction descriptor without N
  uint64_t inv_ctas;     // ceil(2^40 / grid)
  // phase 1
  uint8_t* hq;
  uint8_t* hs;
  const float* h_scale;
  int F;
  // phase 2
  float* y;
  int H;
  int* err;
  int stall;             // failure-detection test: no tokens are loaded until the waits have run out
  uint64_t wait_ns;      // limit of every mbarrier wait
};

// The line of units, in order: active expert, tile along M, token block of the
// expert (so that an expert of more than 64 tokens finds its weights in L2),
// stage of the contraction. A CTA walks from its first unit without divisions.
struct Walk {
  const int4* list;       // active experts: e, first row, rows, first block
  int mt, kb;             // tiles and stages
  int left;               // units still to do
  int a, m, b;            // where the walk stands
  int e, start, n_e, nb;  // of the active expert
  int tile, kb0, kb1;     // the current tile (its index on the line) and its stretch of stages
  int row0, n, slot;      // its token rows

  __device__ __forceinline__ void expert() {
    const int4 x = list[a];
    e = x.x;
    start = x.y;
    n_e = x.z;
    nb = (x.z + kTok - 1) / kTok;
  }
  __device__ __forceinline__ void block() {
    kb1 = min(kb, kb0 + left);
    row0 = start + kTok * b;
    n = min(kTok, n_e - kTok * b);
    slot = start / kTok + b + e;
  }
  __device__ __forceinline__ bool any() const { return left > 0; }
  __device__ __forceinline__ void begin(const int4* l, const int* at, int mt_, int kb_, int units) {
    list = l;
    mt = mt_;
    kb = kb_;
    left = units;
    a = at[0];
    m = at[1];
    b = at[2];
    kb0 = at[3];
    tile = at[4];
    if (left > 0) {
      expert();
      block();
    }
  }
  __device__ __forceinline__ void next() {
    left -= kb1 - kb0;
    kb0 = 0;
    ++tile;
    if (left <= 0) return;
    if (++b == nb) {
      b = 0;
      if (++m == mt) {
        m = 0;
        ++a;
        expert();
      }
    }
    block();
  }
};
// What the stores of a tile need to know of it, and who shares it.
struct Tile {
  int m, row0, n, slot;
  int ca, cb;             // its first and last CTA
};

// The line's U units over G CTAs in grains of one unit, or of a whole tile
// where that makes no stretch more than kWholeSlack units longer than an equal
// share: whole tiles need no partial sums, whose fence (it waits behind the
// weights' copies: 13 to 17 us in mid-walk, 2 at its end), counter and join cost
// more than those units. Slack 0 / 6 / 12 measured 71.8 / 70.0 / 68.9 us on 64
// tokens of the fine-grained NVFP4 layer and 281 / 280 / 277 us on 33 of the
// Scout-shaped blockwise one. `more` CTAs have one grain more than the others.
constexpr int kWholeSlack = 12;
struct Split {
  int G, grain, base, more;
  // n / ctas of a launch: the host's ceil(2^40 / ctas), exact for n below 2^28
  static __device__ __forceinline__ int over(int n, int ctas, uint64_t inv) {
    return static_cast<int>(static_cast<uint64_t>(n) * inv >> 40);
  }
  __device__ __forceinline__ void make(int tiles, int kb, int ctas, uint64_t inv) {
    const int U = tiles * kb;
    const int longest = tiles <= ctas ? kb : over(tiles + ctas - 1, ctas, inv) * kb;
    const int share = U <= ctas ? 1 : over(U + ctas - 1, ctas, inv);
    const bool whole = longest <= share + kWholeSlack;
    grain = whole ? kb : 1;
    const int n = whole ? tiles : U;
    G = max(1, min(ctas, n));
    base = n <= ctas ? min(n, 1) : over(n, ctas, inv);
    more = n - base * G;
  }
  __device__ __forceinline__ int first(int c) const { return grain * (min(c, G) * base + min(c, more)); }
  __device__ __forceinline__ int units(int c) const { return c < G ? grain * (base + (c < more ? 1 : 0)) : 0; }
  __device__ __forceinline__ int owner(int u) const {     // the CTA that has unit u (grains of one)
    const int edge = more * (base + 1);
    return u < edge ? u / (base + 1) : more + (u - edge) / base;
  }
};

// Sum of the 4 columns at `o` of the partial results of CTAs ca..cb, added in
// that order; four CTAs' values are requested together.
__device__ __forceinline__ void join4(const float* part, int64_t place, int ca, int cb, int nc, float* g, float* h) {
#pragma unroll
  for (int j = 0; j < 4; ++j) g[j] = h[j] = 0.0f;
  for (int q0 = ca; q0 <= cb; q0 += 4) {
    float t[4][4][2];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int q = q0 + i;
      const float* o = part + (2 * q + (q == ca ? 1 : 0)) * place;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const bool on = q <= cb && j < nc;
        t[i][j][0] = on ? __ldcg(o + j * 256) : 0.0f;
        t[i][j][1] = on ? __ldcg(o + j * 256 + 128) : 0.0f;
      }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) g[j] += t[i][j][0], h[j] += t[i][j][1];
  }
}

// h = silu(g) u of four tokens (nj of them real, from column c0 on) and one ffn
// row per thread, quantised along the rows: lane = row within a 32-row block, so
// an MX block is one warp, an NVFP4 block half of one, a 1x128 block the four
// warps. Called in a loop over the tile's tokens: the code of all of them
// unrolled did not fit the instruction cache, and its first fetch took up to
// 9 us behind the weights' copies.
template <int KIND>
__device__ __forceinline__ void store_h(const FewArgs& p, const Tile& s, int c0, int nj, float (&g)[4], const float (&u)[4],
                                        float alpha, int row, float sh, int grp, uint32_t (*smax)[4][16], uint32_t& tick) {
  const uint32_t lane = threadIdx.x & 31, wq = row >> 5;
  const int64_t f0 = static_cast<int64_t>(s.m) * 128;
#pragma unroll
  for (int j = 0; j < 4; ++j) g[j] = swiglu_f32(g[j] * alpha, u[j] * alpha);
  if (KIND == kBLK) {
    uint32_t mine = 0;     // lane j keeps token j's maximum over this warp's rows
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const uint32_t m = __reduce_max_sync(0xFFFFFFFFu, __float_as_uint(g[j]) & 0x7FFFFFFFu);
      if (lane == j) mine = m;
    }
    // (two buffers in turn: a warp writes one again only after the barrier
    // that every warp reaches when it has read it)
    ++tick;
    if (lane < 4) smax[tick & 1][wq][4 * grp + lane] = mine;
    group_sync(grp);
  }
  // the four tokens side by side, whether real or not, then the stores
  uint32_t code[4], scale[4];
  float inv[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    uint32_t m = __float_as_uint(g[j]) & 0x7FFFFFFFu;
    scale[j] = 0;
    inv[j] = 0.0f;
    if (KIND == kMX) {
      const int e = mx_exponent(__reduce_max_sync(0xFFFFFFFFu, m), 8, true);
      code[j] = cvt_e4m3x2(__fmul_rn(g[j], mx_multiplier(e)), 0.0f);
      scale[j] = mx_scale_code(e);
    } else if (KIND == kNV) {
#pragma unroll
      for (int o = 8; o > 0; o >>= 1) m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
      scale[j] = cvt_ue4m3(__fmul_rn(__fdiv_rn(__uint_as_float(m), 6.0f), sh));
      const float sc = ue4m3_value(scale[j]);
      const float v = __fmul_rn(g[j], sc == 0.0f ? 0.0f : __fdiv_rn(sh, sc));
      code[j] = cvt_e2m1x2(v, __shfl_down_sync(0xFFFFFFFFu, v, 1));
    } else if (KIND == kBLK) {
      m = 0;
#pragma unroll
      for (int q = 0; q < 4; ++q) m = max(m, smax[tick & 1][q][4 * grp + j]);
      const float mult = blk_scale_few(m);
      inv[j] = __fdiv_rn(1.0f, mult);
      code[j] = cvt_e4m3x2(__fmul_rn(g[j], mult), 0.0f);
    } else {
      code[j] = cvt_e4m3x2(__fmul_rn(g[j], sh), 0.0f);
    }
  }
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    if (j >= nj) break;
    const int col = c0 + j;
    const int64_t r = s.row0 + col;
    const uint32_t in_chunk = (col & 31) * 16 + (col >> 5) * 4;
    if (KIND == kNV) {
      if ((lane & 1) == 0) p.hq[(r * p.F + f0 + row) / 2] = static_cast<uint8_t>(code[j]);
      if ((lane & 15) == 0)
        p.hs[(static_cast<int64_t>(s.slot) * (p.F / 64) + 2 * s.m + (row >> 6)) * 512 + in_chunk + ((row >> 4) & 3)] =
            static_cast<uint8_t>(scale[j]);
    } else {
      p.hq[r * p.F + f0 + row] = static_cast<uint8_t>(code[j]);
      if (KIND == kMX && lane == 0)
        p.hs[(static_cast<int64_t>(s.slot) * (p.F / 128) + s.m) * 512 + in_chunk + wq] = static_cast<uint8_t>(scale[j]);
      if (KIND == kBLK && row == 0)
        reinterpret_cast<float*>(p.hs)[(static_cast<int64_t>(s.slot) * (p.F / 128) + s.m) * kTok + col] = inv[j];
    }
  }
}

__device__ __forceinline__ void store_y(const FewArgs& p, const Tile& s, int c0, int nj, const float (&a)[4],
                                        const float (&b)[4], float alpha, int row) {
  const int64_t m0 = static_cast<int64_t>(s.m) * 256 + row;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    if (j >= nj) break;
    float* d = p.y + static_cast<int64_t>(s.row0 + c0 + j) * p.H + m0;
    d[0] = a[j] * alpha;
    if (m0 + 128 < p.H) d[128] = b[j] * alpha;
  }
}

template <int KIND, int PHASE>
__global__ void __launch_bounds__(kThreads, 1)
    few_gemm_kernel(const __grid_constant__ CUtensorMap tmW, const __grid_constant__ CUtensorMap tmX, const FewArgs p) {
  constexpr uint32_t CH = sf_chunks(KIND), SF = sf_bytes(KIND);
  constexpr bool BS = KIND == kMX || KIND == kNV;      // block scales through tensor memory
  constexpr uint32_t kCols = BS ? 512 : 256;           // two accumulators of 2 x 64 columns, then scale columns
  constexpr int kMost = KIND == kNV ? 5 : kMaxStages;  // NVFP4: 48 scale columns a stage
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = ptx::smem_u32(smem_raw);
  uint8_t* smem = smem_raw + (((raw + 1023u) & ~1023u) - raw);
  // stages first (1024-byte aligned operand tiles), then the small things
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + p.stage_mem);
  uint64_t* full = bars;
  uint64_t* empty = bars + kMaxStages;
  uint64_t* t_full = bars + 2 * kMaxStages;
  uint64_t* t_empty = t_full + 2;
  uint64_t* mma_done = t_empty + 2;                    // after a wait that ran out: no MMA in flight
  uint32_t* s_tmem = reinterpret_cast<uint32_t*>(mma_done + 1);
  volatile int* s_abort = reinterpret_cast<volatile int*>(s_tmem + 1);
  volatile int* s_last = reinterpret_cast<volatile int*>(s_tmem + 2);
  int* s_at = reinterpret_cast<int*>(s_tmem + 4);      // [6] start of the walk, rows of the largest group
  Split* s_split = reinterpret_cast<Split*>(s_tmem + 10);
  uint32_t (*smax)[4][16] = reinterpret_cast<uint32_t (*)[4][16]>(bars + kBars);   // [2][4][16]
  int4* s_list = reinterpret_cast<int4*>(bars + kBars + 64);
  int* s_cnt = reinterpret_cast<int*>(s_list + p.list);

  const int warp = threadIdx.x >> 5;
  const uint32_t lane = threadIdx.x & 31;
  const int cta = blockIdx.x, ctas = gridDim.x;
  grid_launch();
  if (threadIdx.x == 32) {
    for (int s = 0; s < kMost; ++s) {
      ptx::mbar_init(&full[s], 1);
      ptx::mbar_init(&empty[s], KIND == kBLK ? 1 + kEpiWarps : 1);   // the MMAs; BLK: and the epilogue warps
    }
    for (int a = 0; a < 2; ++a) {
      ptx::mbar_init(&t_full[a], 1);
      ptx::mbar_init(&t_empty[a], kEpiWarps);
    }
    ptx::mbar_init(mma_done, 1);
    *s_abort = 0;
    ptx::fence_mbar_init();
    ptx::prefetch_tmap(&tmW);
    ptx::prefetch_tmap(&tmX);
  }
  // rows per expert
  for (int i = threadIdx.x; i < p.E; i += kThreads) s_cnt[i] = 0;
  int e0 = threadIdx.x < p.R ? __ldg(p.idx + threadIdx.x) : -1;
  __syncthreads();
  for (int i = threadIdx.x; i < p.R; i += kThreads) {
    const int e = i < kThreads ? e0 : __ldg(p.idx + i);
    if (e >= 0 && e < p.E) atomicAdd(&s_cnt[e], 1);
  }
  if (warp == 1) {
    __syncwarp();
    ptx::tmem_alloc(s_tmem, kCols);
    ptx::tmem_relinquish();
  }
  __syncthreads();
  if (warp == 0) {
    // The active experts in order. A lane takes a run of experts; one scan
    // gives its first row, block and place (rows and blocks below 2^11 each,
    // places below 2^10).
    const int per = (p.E + 31) / 32, lo = lane * per, hi = min(p.E, lo + per);
    uint32_t mine = 0, most = 0;
    for (int e = lo; e < hi; ++e) {
      const uint32_t n = s_cnt[e];
      most = max(most, n);
      if (n) mine += n | ((n + kTok - 1) / kTok) << 11 | 1u << 22;
    }
    uint32_t sum = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t x = __shfl_up_sync(0xFFFFFFFFu, sum, o);
      if (lane >= o) sum += x;
    }
    const uint32_t all = __shfl_sync(0xFFFFFFFFu, sum, 31);
    most = __reduce_max_sync(0xFFFFFFFFu, most);
    sum -= mine;
    int row = sum & 2047, blk = (sum >> 11) & 2047, at = sum >> 22;
    // this CTA's first unit and the expert it falls in
    Split sp;
    sp.make(static_cast<int>((all >> 11) & 2047) * p.mt, p.kb, ctas, p.inv_ctas);
    const int u0 = sp.first(cta);
    const int tile = sp.grain == 1 ? u0 / p.kb : min(cta, sp.G) * sp.base + min(cta, sp.more);
    for (int e = lo; e < hi; ++e) {
      const int n = s_cnt[e];
      if (n == 0) continue;
      const int nb = (n + kTok - 1) / kTok;
      s_list[at] = make_int4(e, row, n, blk);
      const int local = tile - blk * p.mt;
      if (local >= 0 && local < nb * p.mt) {
        s_at[0] = at;
        s_at[1] = nb == 1 ? local : local / nb;
        s_at[2] = nb == 1 ? 0 : local % nb;
        s_at[3] = u0 - tile * p.kb;
        s_at[4] = tile;
      }
      row += n;
      blk += nb;
      ++at;
    }
    if (lane == 0) {
      s_at[5] = static_cast<int>(most);
      *s_split = sp;
    }
  }
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  const uint32_t tmem = *s_tmem;
  const Split sp = *s_split;
  const int units = sp.units(cta);
  // as many stages as the largest token block of the call leaves room for
  const uint32_t bt = static_cast<uint32_t>((min(s_at[5], kTok) + 15) / 16) * 2048;
  const int STG = min(kMost, static_cast<int>(p.stage_mem / (2 * kATile + bt + SF)));
  uint8_t* sA = smem;
  uint8_t* sB = sA + STG * 2 * kATile;
  uint8_t* sSF = sB + STG * bt;
  Walk s;
  s.begin(s_list, s_at, p.mt, p.kb, units);

  if (warp == 0) {
    if (elect_one()) {
      // ---------------------------------------------------------- producer
      // The weights do not depend on the launch before: the first stages of
      // them are requested before the wait for it, the tokens' after.
      auto load_w = [&](const Walk& s, int kb, int st) {
        const bool two = PHASE == 1 || s.m * 256 + 128 < p.rows_end;
        const int64_t row = s.e * p.rows_e + static_cast<int64_t>(s.m) * p.mstep;
        const uint32_t n16 = (s.n + 15) / 16;
        ptx::mbar_arrive_expect_tx(&full[st], (two ? 2 : 1) * (kATile + CH * 512) + n16 * 2048 +
                                                  (KIND == kBLK ? 256u : CH * 512));
        ptx::tma_load_2d(sA + st * 2 * kATile, &tmW, &full[st], kb * 128, static_cast<int32_t>(row));
        if (two)
          ptx::tma_load_2d(sA + st * 2 * kATile + kATile, &tmW, &full[st], kb * 128,
                           static_cast<int32_t>(row + p.half2));
        if (BS) {
          const uint8_t* f = p.sfa + ((row / 128) * p.sfa_kb4 + static_cast<int64_t>(kb) * CH) * 512;
          ptx::bulk_load(sSF + st * SF, f, CH * 512, &full[st]);
          if (two)
            ptx::bulk_load(sSF + st * SF + CH * 512, f + static_cast<int64_t>(p.half2 / 128) * p.sfa_kb4 * 512, CH * 512,
                           &full[st]);
        }
      };
      auto load_x = [&](const Walk& s, int kb, int st) {
        for (int i = 0; i < (s.n + 15) / 16; ++i)
          ptx::tma_load_2d(sB + st * bt + i * 2048, &tmX, &full[st], kb * 128, s.row0 + 16 * i);
        if (BS)
          ptx::bulk_load(sSF + st * SF + 2 * CH * 512, p.sfb + (static_cast<int64_t>(s.slot) * p.kb + kb) * CH * 512,
                         CH * 512, &full[st]);
        if (KIND == kBLK)
          ptx::bulk_load(sSF + st * SF, p.sfb + (static_cast<int64_t>(s.slot) * p.kb + kb) * 256, 256, &full[st]);
      };
      int early = 0;
      for (Walk v = s; v.any() && early < STG; v.next())
        for (int kb = v.kb0; kb < v.kb1 && early < STG; ++kb, ++early) load_w(v, kb, early);
      grid_wait();
      if (p.stall)
        for (const uint64_t t0 = ptx::globaltimer_ns(); !*s_abort && ptx::globaltimer_ns() - t0 < 4 * p.wait_ns;) {
        }
      int it = 0, st = 0;
      uint32_t ph = 1;                    // (a first pass over the ring waits for nothing)
      for (; s.any(); s.next()) {
        for (int kb = s.kb0; kb < s.kb1; ++kb, ++it) {
          if (it >= early) {
            if (*s_abort) break;
            if (!ptx::mbar_wait(&empty[st], ph, p.wait_ns)) {
              report(p.err, MGQ_ERR_TIMEOUT);
              *s_abort = 1;
              break;
            }
            load_w(s, kb, st);
          }
          load_x(s, kb, st);
          if (++st == STG) st = 0, ph ^= 1;
        }
        if (*s_abort && it >= early) break;
      }
      // given up: no copy of this CTA may land after it has left (the stages
      // requested early got their tokens too: their barriers can complete)
      if (*s_abort)
        for (int i = it > STG ? it - STG : 0; i < it; ++i)
          ptx::mbar_wait(&full[i % STG], (i / STG) & 1, p.wait_ns / 100);
    }
  } else if (warp == 1) {
    if (elect_one()) {
      // ---------------------------------------------------------- MMA issuer
      const uint32_t sA0 = ptx::smem_u32(sA), sB0 = ptx::smem_u32(sB), sF0 = ptx::smem_u32(sSF);
      int st = 0;
      uint32_t ph = 0, tc = 0;
      bool ok = true;
      for (; s.any() && ok; s.next()) {
        const bool two = PHASE == 1 || s.m * 256 + 128 < p.rows_end;
        const uint32_t idesc = p.idesc0 | (static_cast<uint32_t>((s.n + 15) / 16 * 2) << 17);
        uint32_t a = tc & 1;
        for (int kb = s.kb0; kb < s.kb1; ++kb) {
          if (KIND == kBLK || kb == s.kb0) {
            a = tc & 1;
            ok = !*s_abort && ptx::mbar_wait(&t_empty[a], ((tc >> 1) & 1) ^ 1, p.wait_ns);
          }
          ok = ok && !*s_abort && ptx::mbar_wait(&full[st], ph, p.wait_ns);
          if (!ok) {
            report(p.err, MGQ_ERR_TIMEOUT);
            *s_abort = 1;
            break;
          }
          ptx::tc_fence_after();
          const uint32_t sf_t = tmem + 256 + st * 12 * CH;
          if constexpr (BS) {
#pragma unroll
            for (uint32_t c = 0; c < CH; ++c) {
              ptx::tmem_cp_32x128b_x4(sf_t + c * 4, ptx::sdesc_sf(sF0 + st * SF + c * 512));
              if (two) ptx::tmem_cp_32x128b_x4(sf_t + (CH + c) * 4, ptx::sdesc_sf(sF0 + st * SF + (CH + c) * 512));
              ptx::tmem_cp_32x128b_x4(sf_t + (2 * CH + c) * 4, ptx::sdesc_sf(sF0 + st * SF + (2 * CH + c) * 512));
            }
          }
          const uint64_t bd = ptx::sdesc_kmajor_sw128(sB0 + st * bt);
          const uint64_t ad = ptx::sdesc_kmajor_sw128(sA0 + st * 2 * kATile);
#pragma unroll
          for (int kk = 0; kk < 4; ++kk) {
            const uint32_t acc = ((KIND != kBLK && kb > s.kb0) || kk > 0) ? 1u : 0u;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              if (h == 1 && !two) break;
              const uint64_t adk = ad + h * (kATile >> 4) + kk * 2;
              const uint32_t d = tmem + a * 2 * kTok + h * kTok;
              if (KIND == kNV)
                ptx::mma_mxf4nvf4(d, adk, bd + kk * 2, idesc, sf_t + (h * CH + kk) * 4, sf_t + (2 * CH + kk) * 4, acc);
              else if (KIND == kMX)
                ptx::mma_mxf8f6f4(d, adk, bd + kk * 2, idesc | ptx::idesc_sf_ids(kk, kk), sf_t + h * 4, sf_t + 8, acc);
              else
                ptx::mma_f8f6f4(d, adk, bd + kk * 2, idesc, acc);
            }
          }
          ptx::mma_commit(&empty[st]);
          if (KIND == kBLK || kb == s.kb1 - 1) {
            ptx::mma_commit(&t_full[a]);
            ++tc;
          }
          if (++st == STG) st = 0, ph ^= 1;
        }
      }
      if (*s_abort) {
        ptx::mma_commit(mma_done);
        ptx::mbar_wait(mma_done, 0, p.wait_ns / 100);
      }
    }
  } else {
    // ------------------------------------------------------------ epilogue
    // thread = one weight row of each half (tensor-memory lane) and half of the
    // tokens: the groups take four columns in turn (1x128: sixteen)
    grid_wait();
    const int row = (warp & 3) * 32 + lane, grp = (warp - 2) >> 2;
    const uint32_t tlane = static_cast<uint32_t>(warp & 3) << 21;
    const int64_t place = static_cast<int64_t>(p.nmax) * 256;
    const float sx = KIND == kNV || KIND == kTEN ? __ldg(p.sx) : 1.0f;
    const float sh = PHASE == 1 && (KIND == kNV || KIND == kTEN) ? __ldg(p.h_scale) : 1.0f;
    int st = 0;
    uint32_t ph = 0, tc = 0, tick = 0;
    bool alive = true;
    for (; s.any(); s.next()) {
      const int n16 = (s.n + 15) / 16;
      const bool whole = s.kb1 - s.kb0 == p.kb;
      float alpha = 1.0f;
      if (KIND == kNV || KIND == kTEN) alpha = 1.0f / (sx * __ldg(p.sw + s.e));
      Tile t{s.m, s.row0, s.n, s.slot, 0, 0};
      // this CTA's place for partial sums: the second for its last tile (and,
      // before that, 1x128 whole ones), the first for one begun by another CTA
      float* mine = p.part + (2 * cta + 1) * place;
      if (!whole) {
        const int first = s.tile * p.kb;
        t.ca = sp.owner(first);
        t.cb = sp.owner(first + p.kb - 1);
        if (t.ca != cta) mine -= place;
      }
      if (KIND == kBLK) {
        // every stage's product is scaled and added in float32 registers
        float acc[2][kTok / 32][16];
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int c = 0; c < kTok / 32; ++c)
#pragma unroll
            for (int j = 0; j < 16; ++j) acc[h][c][j] = 0.0f;
        const int64_t wr = (s.e * p.rows_e + static_cast<int64_t>(s.m) * p.mstep) / 128;
        const bool two = PHASE == 1 || s.m * 256 + 128 < p.rows_end;
        float w0v = 0.0f, w1v = 0.0f;
        for (int kb = s.kb0; kb < s.kb1; ++kb, ++tc) {
          const uint32_t a = tc & 1;
          if (((kb - s.kb0) & 31) == 0) {      // the weight scales of the next 32 stages, one a lane
            const int k = min(kb + static_cast<int>(lane), s.kb1 - 1);
            w0v = __ldg(p.sw + wr * p.kblk + k);
            w1v = two ? __ldg(p.sw + (wr + p.half2 / 128) * p.kblk + k) : 0.0f;
          }
          const float w0 = __shfl_sync(0xFFFFFFFFu, w0v, (kb - s.kb0) & 31);
          const float w1 = __shfl_sync(0xFFFFFFFFu, w1v, (kb - s.kb0) & 31);
          alive = __all_sync(0xFFFFFFFFu, !*s_abort && ptx::mbar_wait(&full[st], ph, p.wait_ns) &&
                                              ptx::mbar_wait(&t_full[a], (tc >> 1) & 1, p.wait_ns));
          if (!alive) break;
          ptx::tc_fence_after();
          const float4* fx = reinterpret_cast<const float4*>(sSF + st * SF);
#pragma unroll
          for (int c = 0; c < kTok / 32; ++c) {
            const int c16 = 2 * c + grp;
            if (c16 >= n16) break;
            uint32_t v0[16], v1[16];
            ptx::tmem_ld_32x32b_x16(tmem + tlane + a * 2 * kTok + 16 * c16, v0);
            ptx::tmem_ld_32x32b_x16(tmem + tlane + a * 2 * kTok + kTok + 16 * c16, v1);
            ptx::tmem_ld_wait_regs(v0);
            ptx::tmem_ld_wait_regs(v1);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const float4 f = fx[4 * c16 + j];
              const float f4[4] = {f.x, f.y, f.z, f.w};
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                acc[0][c][4 * j + i] = fmaf(__uint_as_float(v0[4 * j + i]), f4[i] * w0, acc[0][c][4 * j + i]);
                if (two) acc[1][c][4 * j + i] = fmaf(__uint_as_float(v1[4 * j + i]), f4[i] * w1, acc[1][c][4 * j + i]);
              }
            }
          }
          ptx::tc_fence_before();
          __syncwarp();
          if (lane == 0) {
            ptx::mbar_arrive(&t_empty[a]);
            ptx::mbar_arrive(&empty[st]);
          }
          if (++st == STG) st = 0, ph ^= 1;
        }
        // the sums go to this CTA's place even for a whole tile, whose threads
        // read back what they wrote: registers cannot be walked in a loop
        alive = epi_all(alive);            // (store_h has barriers of its own)
        if (alive) {
#pragma unroll
          for (int c = 0; c < kTok / 32; ++c) {
            const int c0 = 32 * c + 16 * grp;
            if (c0 >= s.n) break;
#pragma unroll
            for (int j = 0; j < 16; ++j) {
              if (c0 + j >= s.n) break;
              mine[(c0 + j) * 256 + row] = acc[0][c][j];
              mine[(c0 + j) * 256 + 128 + row] = acc[1][c][j];
            }
          }
          if (whole) {
#pragma unroll 1
            for (int c = 16 * grp; c < s.n; c += (c & 12) == 12 ? 20 : 4) {
              const int nj = min(4, s.n - c);
              float g[4], h[4];
#pragma unroll
              for (int j = 0; j < 4; ++j) {
                g[j] = j < nj ? mine[(c + j) * 256 + row] : 0.0f;
                h[j] = j < nj ? mine[(c + j) * 256 + 128 + row] : 0.0f;
              }
              if (PHASE == 1) store_h<KIND>(p, t, c, nj, g, h, alpha, row, sh, grp, smax, tick);
              else store_y(p, t, c, nj, g, h, alpha, row);
            }
          }
        }
      } else {
        const uint32_t a = tc & 1;
        alive = epi_all(!*s_abort && ptx::mbar_wait(&t_full[a], (tc >> 1) & 1, p.wait_ns));
        ++tc;
        if (alive) {
          ptx::tc_fence_after();
#pragma unroll 1
          for (int c = 4 * grp; c < s.n; c += 8) {
            const int nj = min(4, s.n - c);
            uint32_t v0[4], v1[4];
            ptx::tmem_ld_32x32b_x4(tmem + tlane + a * 2 * kTok + c, v0);
            ptx::tmem_ld_32x32b_x4(tmem + tlane + a * 2 * kTok + kTok + c, v1);
            ptx::tmem_ld_wait_regs2(v0, v1);
            float g[4], h[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) g[j] = __uint_as_float(v0[j]), h[j] = __uint_as_float(v1[j]);
            if (!whole) {
#pragma unroll
              for (int j = 0; j < 4; ++j) {
                if (j >= nj) break;
                mine[(c + j) * 256 + row] = g[j];
                mine[(c + j) * 256 + 128 + row] = h[j];
              }
            } else if (PHASE == 1) {
              store_h<KIND>(p, t, c, nj, g, h, alpha, row, sh, grp, smax, tick);
            } else {
              store_y(p, t, c, nj, g, h, alpha, row);
            }
          }
          ptx::tc_fence_before();
          __syncwarp();
          if (lane == 0) ptx::mbar_arrive(&t_empty[a]);
        }
      }
      if (!alive) {                        // (in all the warps)
        report(p.err, MGQ_ERR_TIMEOUT);
        *s_abort = 1;
        break;
      }
      if (!whole) {
        // the barrier orders the warps' stores before the fence of the
        // thread that counts this CTA in
        epi_sync();
        if (threadIdx.x == 64) {
          __threadfence();
          *s_last = atomicAdd(p.cnt + t.ca, 1) == t.cb - t.ca;
          __threadfence();
        }
        epi_sync();
        if (*s_last) {
#pragma unroll 1
          for (int c = 4 * grp; c < t.n; c += 8) {
            const int nj = min(4, t.n - c);
            float g[4], h[4];
            join4(p.part + c * 256 + row, place, t.ca, t.cb, nj, g, h);
            if (PHASE == 1) store_h<KIND>(p, t, c, nj, g, h, alpha, row, sh, grp, smax, tick);
            else store_y(p, t, c, nj, g, h, alpha, row);
          }
        }
      }
    }
  }
  ptx::tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    __syncwarp();
    ptx::tc_fence_after();
    ptx::tmem_dealloc(tmem, kCols);
  }
}

// out[t] = sum_j probs[t, j] y[row(t, j)] in float32, j ascending, rounded once
__global__ void __launch_bounds__(128) few_combine_kernel(const float* y, const int32_t* row_of, const float* probs, int T,
                                                          int k, int H, uint16_t* out) {
  grid_launch();
  grid_wait();
  const int t = blockIdx.y, c = (blockIdx.x * 128 + threadIdx.x) * 4;
  if (c >= H) return;
  // all rows requested before the first is used; added in the order of j
  float4 v[kMaxK];
  float pr[kMaxK];
#pragma unroll
  for (int j = 0; j < kMaxK; ++j) {
    const int r = j < k ? row_of[t * k + j] : -1;
    pr[j] = r >= 0 ? __ldg(probs + t * k + j) : 0.0f;
    v[j] = r >= 0 ? *reinterpret_cast<const float4*>(y + static_cast<int64_t>(r) * H + c) : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  }
  float4 o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
  for (int j = 0; j < kMaxK; ++j) {
    o.x = fmaf(pr[j], v[j].x, o.x);
    o.y = fmaf(pr[j], v[j].y, o.y);
    o.z = fmaf(pr[j], v[j].z, o.z);
    o.w = fmaf(pr[j], v[j].w, o.w);
  }
  *reinterpret_cast<uint2*>(out + static_cast<int64_t>(t) * H + c) =
      make_uint2(pack_bf16x2(o.x, o.y), pack_bf16x2(o.z, o.w));
}

// ---------------------------------------------------------------------------
// host side

int kind_of(int scaling) {
  switch (scaling) {
    case MGQ_MX32_E8M0: return kMX;
    case MGQ_NV16_UE4M3: return kNV;
    case MGQ_BLK_1x128_F32: return kBLK;
    case MGQ_TENSOR_F32: return kTEN;
    default: return -1;
  }
}

bool few_sizes_ok(int T, int k, int E, int64_t H, int64_t F, int kind) {
  const int64_t unit = kind == kNV ? 256 : 128;
  return T >= 0 && T <= kMaxT && k >= 1 && k <= kMaxK && E >= 1 && E <= kMaxE && k <= E && H >= unit && F >= unit &&
         H % unit == 0 && F % unit == 0 && H <= 65536 && F <= 65536;
}

struct Layout {
  int64_t row_of, cnt, xq, xs, hq, hs, y, part, total;
  int nmax, grid;
};

Layout layout_of(int T, int k, int E, int64_t H, int64_t F, int kind) {
  Layout l{};
  const int64_t R = static_cast<int64_t>(T) * k, slots = R / kTok + E;
  // (a token may name an expert more than once: up to R rows, not T, of one expert)
  l.nmax = static_cast<int>((R < kTok ? R + 15 : kTok) / 16 * 16);
  l.grid = num_sms();
  const int64_t per = kind == kNV ? 2 : 1;                      // codes per byte
  auto scales = [&](int64_t K) {
    return kind == kMX ? slots * (K / 128) * 512 : kind == kNV ? slots * (K / 64) * 512 :
           kind == kBLK ? slots * (K / 128) * 256 : int64_t(0);
  };
  int64_t at = 0;
  auto take = [&](int64_t bytes) {
    const int64_t o = at;
    at += (bytes + 255) / 256 * 256;
    return o;
  };
  l.row_of = take(R * 4);
  l.cnt = take(2 * l.grid * 4);
  l.xq = take(R * H / per);
  l.xs = take(scales(H));
  l.hq = take(R * F / per);
  l.hs = take(scales(F));
  l.y = take(R * H * 4);
  l.part = take(2 * static_cast<int64_t>(l.grid) * l.nmax * 256 * 4);
  l.total = at;
  return l;
}

constexpr size_t kSmemMax = 227 * 1024;

template <int KIND, int PHASE>
int launch_gemm(const CUtensorMap& tw, const CUtensorMap& tx, FewArgs p, int grid, cudaStream_t s) {
  auto kern = few_gemm_kernel<KIND, PHASE>;
  static bool attr_set[64] = {false};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return MGQ_ERR_CUDA;
  if (dev >= 64 || !attr_set[dev]) {
    if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(kSmemMax)) != cudaSuccess)
      return MGQ_ERR_CUDA;
    if (dev < 64) attr_set[dev] = true;
  }
  // what is not a stage: alignment, barriers and flags, block maxima, the
  // list of active experts, the counts
  const size_t small = kBars * 8 + 128 * 4 + static_cast<size_t>(p.list) * 16 + static_cast<size_t>(p.E) * 4;
  p.stage_mem = static_cast<uint32_t>((kSmemMax - 1024 - small) / 1024 * 1024);
  return launch_after(kern, dim3(grid), kThreads, 1024 + p.stage_mem + small, 1, s, tw, tx, p) ? MGQ_OK : MGQ_ERR_CUDA;
}

template <int KIND>
int few_forward(const void* x, int T, int64_t H, int64_t F, const int32_t* idx, const float* probs, int k, int E,
                const mgq_operand* W1, const mgq_operand* W2, const float* x_scale, const float* h_scale, void* out,
                uint8_t* ws, cudaStream_t s) {
  const Layout l = layout_of(T, k, E, H, F, KIND);
  const int R = T * k;
  const int64_t per = KIND == kNV ? 2 : 1;
  CUtensorMap tw1, tw2, tx, th;
  if (!encode_tmap_u8_2d(&tw1, W1->data, H / per, static_cast<uint64_t>(E) * 2 * F, W1->ld / per, 128, 128) ||
      !encode_tmap_u8_2d(&tw2, W2->data, F / per, static_cast<uint64_t>(E) * H, W2->ld / per, 128, 128) ||
      !encode_tmap_u8_2d(&tx, ws + l.xq, H / per, R, H / per, 128, 16) ||
      !encode_tmap_u8_2d(&th, ws + l.hq, F / per, R, F / per, 128, 16))
    return MGQ_ERR_CUDA;
  int* err = error_word();

  PrepArgs pa{};
  pa.x = static_cast<const uint16_t*>(x);
  pa.idx = idx;
  pa.R = R;
  pa.k = k;
  pa.E = E;
  pa.H = static_cast<int>(H);
  pa.xq = ws + l.xq;
  pa.xs = ws + l.xs;
  pa.x_scale = x_scale;
  pa.row_of = reinterpret_cast<int32_t*>(ws + l.row_of);
  pa.cnt = reinterpret_cast<int32_t*>(ws + l.cnt);
  pa.ncnt = 2 * l.grid;
  pa.err = err;
  const int warps = R * static_cast<int>((H + 1023) / 1024);
  if (!launch_after(few_prep_kernel<KIND>, dim3((warps + 3) / 4), 128, 0, 1, s, pa)) return MGQ_ERR_CUDA;

  FewArgs a{};
  a.idx = idx;
  a.R = R;
  a.E = E;
  a.part = reinterpret_cast<float*>(ws + l.part);
  a.nmax = l.nmax;
  a.list = E < R ? E : R;
  a.inv_ctas = ((uint64_t(1) << 40) + l.grid - 1) / l.grid;
  a.err = err;
  debug_knobs(&a.stall, &a.wait_ns);
  a.hq = ws + l.hq;
  a.hs = ws + l.hs;
  a.h_scale = h_scale;
  a.F = static_cast<int>(F);
  a.y = reinterpret_cast<float*>(ws + l.y);
  a.H = static_cast<int>(H);
  a.idesc0 = KIND == kNV ? ptx::idesc_mxf4nvf4_ue4m3(128, 0) : KIND == kMX ? ptx::idesc_mxf8f6f4(0, 0, 128, 0)
                                                              : ptx::idesc_f8f6f4(0, 0, 128, 0);
  auto weight = [&](const mgq_operand* W) {
    a.sfa = static_cast<const uint8_t*>(W->scale);
    a.sfa_kb4 = W->ld / (KIND == kNV ? 64 : 128);
    a.sw = KIND == kNV ? W->global_scale : static_cast<const float*>(W->scale);
  };
  // gate and up
  a.rows_e = 2 * F;
  a.mt = static_cast<int>(F / 128);
  a.kb = static_cast<int>(H / per / 128);
  a.kblk = static_cast<int>(H / 128);
  a.half2 = static_cast<int>(F);
  a.mstep = 128;
  a.sfb = ws + l.xs;
  a.sx = x_scale;
  a.cnt = reinterpret_cast<int32_t*>(ws + l.cnt);
  weight(W1);
  int rc = launch_gemm<KIND, 1>(tw1, tx, a, l.grid, s);
  if (rc != MGQ_OK) return rc;
  // down
  a.rows_e = H;
  a.rows_end = static_cast<int>(H);
  a.mt = static_cast<int>((H + 255) / 256);
  a.kb = static_cast<int>(F / per / 128);
  a.kblk = static_cast<int>(F / 128);
  a.half2 = 128;
  a.mstep = 256;
  a.sfb = ws + l.hs;
  a.sx = h_scale;
  a.cnt += l.grid;
  weight(W2);
  rc = launch_gemm<KIND, 2>(tw2, th, a, l.grid, s);
  if (rc != MGQ_OK) return rc;
  return launch_after(few_combine_kernel, dim3((H + 511) / 512, T), 128, 0, 1, s, static_cast<const float*>(a.y),
                      static_cast<const int32_t*>(pa.row_of), probs, T, k, static_cast<int>(H),
                      static_cast<uint16_t*>(out))
             ? MGQ_OK
             : MGQ_ERR_CUDA;
}

}  // namespace
}  // namespace mgq

using namespace mgq;

extern "C" size_t mgq_moe_few_workspace_size(int T, int k, int E, int64_t H, int64_t F, int scaling) {
  const int kind = kind_of(scaling);
  if (kind < 0 || !few_sizes_ok(T, k, E, H, F, kind)) return 0;
  if (few_is_small(kind, T, k, E, H, F)) return few_small_workspace(T, k, F, kind);
  return static_cast<size_t>(layout_of(T, k, E, H, F, kind).total);
}

extern "C" int mgq_moe_few_forward(const void* x_bf16, int T, int64_t H, int64_t F, const int32_t* topk_idx,
                                   const float* probs, int k, int E, const mgq_operand* W1, const mgq_operand* W2,
                                   int scaling, const float* x_scale, const float* h_scale, void* out_bf16,
                                   void* workspace, size_t ws_bytes, void* stream) {
  MGQ_CHECK_ARG(W1 && W2);
  const int kind = kind_of(scaling);
  if (kind < 0) return MGQ_ERR_UNSUPPORTED;
  const int dt = kind == kNV ? MGQ_E2M1 : MGQ_E4M3;
  if (W1->dtype != dt || W2->dtype != dt) return MGQ_ERR_UNSUPPORTED;
  if (W1->layout != MGQ_LAYOUT_K || W2->layout != MGQ_LAYOUT_K) return MGQ_ERR_UNSUPPORTED;
  MGQ_CHECK_ARG(few_sizes_ok(T, k, E, H, F, kind));
  if (T == 0) return MGQ_OK;
  MGQ_CHECK_ARG(x_bf16 && topk_idx && probs && out_bf16 && workspace);
  MGQ_CHECK_ARG(aligned16(x_bf16) && aligned16(out_bf16) && (reinterpret_cast<uintptr_t>(workspace) & 255) == 0);
  for (const mgq_operand* W : {W1, W2}) {
    const int64_t K = W == W1 ? H : F;
    MGQ_CHECK_ARG(W->data && W->scale && aligned16(W->data));
    // (block scale bytes are copied in vectors, float32 scales read one by one)
    MGQ_CHECK_ARG((reinterpret_cast<uintptr_t>(W->scale) & (kind == kMX || kind == kNV ? 15 : 3)) == 0);
    MGQ_CHECK_ARG(W->ld >= K && W->ld % (kind == kNV ? 256 : 128) == 0);
    if (kind == kNV) MGQ_CHECK_ARG(W->global_scale);
    if (kind == kBLK) MGQ_CHECK_ARG(W->ld == K);          // 128x128 scales are laid out by K
  }
  if (kind == kNV || kind == kTEN) MGQ_CHECK_ARG(x_scale && h_scale);
  MGQ_CHECK_ARG(ws_bytes >= mgq_moe_few_workspace_size(T, k, E, H, F, scaling));
  cudaStream_t s = as_stream(stream);
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  if (few_is_small(kind, T, k, E, H, F))
    return few_small_forward(kind, x_bf16, T, H, F, topk_idx, probs, k, E, W1, W2, x_scale, h_scale, out_bf16, ws, s);
  switch (kind) {
    case kMX:
      return few_forward<kMX>(x_bf16, T, H, F, topk_idx, probs, k, E, W1, W2, x_scale, h_scale, out_bf16, ws, s);
    case kNV:
      return few_forward<kNV>(x_bf16, T, H, F, topk_idx, probs, k, E, W1, W2, x_scale, h_scale, out_bf16, ws, s);
    case kBLK:
      return few_forward<kBLK>(x_bf16, T, H, F, topk_idx, probs, k, E, W1, W2, x_scale, h_scale, out_bf16, ws, s);
    default:
      return few_forward<kTEN>(x_bf16, T, H, F, topk_idx, probs, k, E, W1, W2, x_scale, h_scale, out_bf16, ws, s);
  }
}
