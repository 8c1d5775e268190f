// What the products over ragged groups share: their arguments, the order of
// their tiles, the groups' offsets, and the stores of token rows from an
// accumulator that holds channels as lanes and tokens as columns.
#pragma once
#include "device_common.cuh"
#include "mgq_internal.h"
#include "ptx_sm100.cuh"

namespace mgq {

struct RaggedArgs {
  const int32_t* offsets;   // [E + 1], or null: one group of all R rows
  int E;
  int64_t R;
  int64_t M;                // fwd, dgrad: output columns; wgrad: rows of an expert's result
  int64_t C;                // fwd, dgrad: length of the contraction; wgrad: columns of the result
  void* out;
  int64_t ldo;              // fwd, dgrad: row pitch of the result
  int out_f32;
  float beta;
  int bk;                   // elements of the contraction a stage
  const float* sx;          // int8: scale of each row, and of each of the E x M channels
  const float* sw;
  int stall;                // failure-detection test: no loads are issued
  uint64_t wait_ns;
  int* err;
};

namespace {

enum { kFwd = 0, kDgrad = 1, kWgrad = 2 };

constexpr int kTile = 256;                         // M side, and tokens (wgrad: columns) at most
constexpr int kMaxE = 1024;
constexpr uint32_t kSmallBox = 32;                 // rows of the token boxes of a group's last tile

struct RaggedTile {
  int e, nst;               // group, contraction stages
  int row0, n;              // fwd, dgrad: first token and tokens of the tile; wgrad: of the group
  int64_t m0, c0;           // first row on the M side; wgrad: first column
};

// Order of the tiles of one group: bands of 8 along the M side (wgrad: along the
// columns), inside a band the band's tiles fastest. A wave of tiles then covers
// a block of about 8 x 9 and finds both operands' re-reads in L2.
__device__ __forceinline__ void banded(int64_t local, int64_t slow, int64_t nfast, int64_t& fast, int64_t& s) {
  constexpr int64_t kBand = 8;
  const int64_t band = local / (kBand * slow), r = local - band * (kBand * slow);
  const int64_t w = min(kBand, nfast - band * kBand);
  s = r / w;
  fast = band * kBand + (r - s * w);
}

template <int OP, int TOK = kTile>
__device__ __forceinline__ bool ragged_tile(const int32_t* s_off, const int32_t* s_cum, const RaggedArgs& p, int64_t t,
                                            int& ecur, RaggedTile& tl) {
  const int64_t nM = (p.M + kTile - 1) / kTile;
  if (OP == kWgrad) {
    const int64_t nC = (p.C + kTile - 1) / kTile, per = nM * nC;
    if (t >= per * p.E) return false;
    const int e = (int)(t / per);
    int64_t c, m;
    banded(t - e * per, nM, nC, c, m);
    tl.e = e;
    tl.row0 = s_off[e];
    tl.n = s_off[e + 1] - s_off[e];
    tl.nst = (tl.n + p.bk - 1) / p.bk;
    tl.m0 = m * kTile;
    tl.c0 = c * kTile;
  } else {
    if (t >= s_cum[p.E] * nM) return false;
    while (ecur < p.E - 1 && s_cum[ecur + 1] * nM <= t) ++ecur;
    const int e = ecur;
    int64_t m, tk;
    banded(t - s_cum[e] * nM, s_cum[e + 1] - s_cum[e], nM, m, tk);
    tl.e = e;
    tl.row0 = s_off[e] + (int)tk * TOK;
    tl.n = min(TOK, s_off[e + 1] - tl.row0);
    tl.nst = (int)((p.C + p.bk - 1) / p.bk);
    tl.m0 = m * kTile;
    tl.c0 = 0;
  }
  return true;
}

// Offsets into shared memory with the running count of token tiles (of TOK tokens), by
// one warp; true if they are a row partition (not negative, not decreasing, within R).
template <int TOK = kTile>
__device__ __forceinline__ bool load_groups(const RaggedArgs& p, int32_t* s_off, int32_t* s_cum, uint32_t lane) {
  int cum = 0;
  bool ok = true;
  for (int b = 0; b < p.E; b += 32) {
    const int e = b + (int)lane;
    const bool in = e < p.E;
    const int lo = in && p.offsets ? p.offsets[e] : 0;
    const int hi = !in ? 0 : p.offsets ? p.offsets[e + 1] : (int)p.R;
    ok &= !in || (lo >= 0 && lo <= hi && hi <= p.R);
    const int mine = in && lo <= hi ? (hi - lo + TOK - 1) / TOK : 0;
    int inc = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xFFFFFFFFu, inc, o);
      if (lane >= o) inc += v;
    }
    if (in) {
      s_off[e] = lo;
      s_cum[e] = cum + inc - mine;
      if (e == p.E - 1) {
        s_off[p.E] = hi;
        s_cum[p.E] = cum + inc;
      }
    }
    cum += __shfl_sync(0xFFFFFFFFu, inc, 31);
  }
  return __all_sync(0xFFFFFFFFu, ok);
}

// 8 x 8 transposition among groups of 8 lanes: v[j] of lane l is (row l, column
// j); the result is row pairs in words, o[i] = rows 2i, 2i + 1 of column l & 7,
// rounded to bf16.
__device__ __forceinline__ uint4 transpose8_bf16(const float* v, uint32_t lane) {
  const bool b0 = lane & 1, b1 = lane & 2, b2 = lane & 4;
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float other = __shfl_xor_sync(0xFFFFFFFFu, b0 ? v[2 * i] : v[2 * i + 1], 1);
    w[i] = b0 ? pack_bf16x2(other, v[2 * i + 1]) : pack_bf16x2(v[2 * i], other);
  }
  uint32_t q[2][2];
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    const uint32_t other = __shfl_xor_sync(0xFFFFFFFFu, b1 ? w[2 * j] : w[2 * j + 1], 2);
    q[j][0] = b1 ? other : w[2 * j];
    q[j][1] = b1 ? w[2 * j + 1] : other;
  }
  const uint32_t o0 = __shfl_xor_sync(0xFFFFFFFFu, b2 ? q[0][0] : q[1][0], 4);
  const uint32_t o1 = __shfl_xor_sync(0xFFFFFFFFu, b2 ? q[0][1] : q[1][1], 4);
  return b2 ? make_uint4(o0, o1, q[1][0], q[1][1]) : make_uint4(q[0][0], q[0][1], o0, o1);
}

// NT tokens of a warp's 32 channels: v[j] = (channel chan0 + lane, token tok0 + j).
// `left` tokens exist.
template <bool F32, int NT>
__device__ __forceinline__ void store_tokens(void* out, int64_t ldo, const float (&v)[NT], int64_t tok0, int left,
                                             int64_t chan0, int64_t chans, uint32_t lane) {
  if (F32) {
    float* o = static_cast<float*>(out) + tok0 * ldo + chan0 + lane;
    const bool in = chan0 + lane < chans;
#pragma unroll
    for (int j = 0; j < NT; ++j)
      if (in && j < left) o[j * ldo] = v[j];
  } else {
    const int64_t c = chan0 + (lane & 24);
    uint16_t* o = static_cast<uint16_t*>(out) + (tok0 + (lane & 7)) * ldo + c;
#pragma unroll
    for (int j = 0; j < NT; j += 8) {
      if (j >= left) break;                                // the same in the whole warp
      const uint4 w = transpose8_bf16(v + j, lane);
      if (j + (int)(lane & 7) < left && c < chans) *reinterpret_cast<uint4*>(o + j * ldo) = w;
    }
  }
}

// The same 32 tokens through shared memory and the TMA, for a run of tokens that
// all belong to the group: a warp's 2 KB slot takes 32 tokens of 32 bf16 channels
// or 16 of float32, in the swizzle of the map. Whole rows of 64 or 128 bytes leave
// without the warp's waiting for the memory: 256 x 256 tiles of a contraction of 64
// took 4.5 us a tile (bf16) and 7.2 (float32) with stores from registers.
constexpr uint32_t kTokSlot = 2048;
template <bool F32>
__device__ __forceinline__ void send_tokens(const CUtensorMap* map, uint8_t* slot, const float (&v)[32], int32_t tok0,
                                            int32_t chan0, uint32_t lane) {
  constexpr int NT = F32 ? 16 : 32;
#pragma unroll
  for (int h = 0; h < 32; h += NT) {
    if (lane == 0) ptx::bulk_wait_read0();                 // the store before has read the slot
    __syncwarp();
#pragma unroll
    for (int j = 0; j < NT; j += 2) {
      if (F32) {
#pragma unroll
        for (int i = j; i < j + 2; ++i)
          *reinterpret_cast<float*>(slot + i * 128 + (((lane >> 2) ^ (i & 7)) << 4) + (lane & 3) * 4) = v[h + i];
      } else {
        const uint32_t w = pack_bf16x2(v[j], v[j + 1]);
        uint8_t* at = slot + j * 64 + (((lane >> 3) ^ ((j >> 1) & 3)) << 4) + (lane & 7) * 2;
        *reinterpret_cast<uint16_t*>(at) = (uint16_t)w;
        *reinterpret_cast<uint16_t*>(at + 64) = (uint16_t)(w >> 16);
      }
    }
    ptx::fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0) {
      ptx::tma_store_3d(map, slot, chan0, tok0 + h, 0);
      ptx::bulk_commit();
    }
  }
}

}  // namespace

// The form for few rows a group (ragged_few.cu); op kFwd or kDgrad, tensor maps of
// the weights and of the rows (boxes of kFewBox rows).
constexpr int kFewBox = 16;
// the map that send_tokens stores with
inline bool encode_out(CUtensorMap* map, void* out, int64_t R, int64_t M, int64_t ldo, bool f32) {
  const uint64_t u = f32 ? 4 : 2;
  return encode_tmap_swz_3d(map, out, (int)u, {(uint64_t)M, (uint64_t)R, 1}, ldo * u, R * ldo * u, {32, f32 ? 16u : 32u, 1});
}
int run_few(int op, bool i8, const CUtensorMap& ta, const CUtensorMap& tb, const RaggedArgs& p, cudaStream_t s);

// The most tiles of `per` tokens that R rows in E groups can need.
inline int64_t token_tiles(int E, int64_t R, int64_t per) {
  const int64_t g = R < E ? R : E;
  return (R - g) / per + g;
}

// Whether a product of R rows over E groups, M output channels, takes that form: up
// to 32 rows a group on average (40 in the GPU's first three waves of tiles), where
// the weights' bytes count and two CTAs an SM stream them best, or so few tiles that
// they fit the GPU at once, where its smaller tiles and the split contraction use
// more SMs. Measured both ways (replayed graphs): 2 rows of 8 experts 4096 x 14336,
// 39 us against 48; 512 rows over 8 x [512, 4096] 8 against 24; 64 x [4096, 4096] with
// 24, 40, 64 and 128 rows each 315, 319, 326 and 399 against 328, 331, 335 and 345; 40
// rows each within three waves 0.78 (contraction of 512) to 1.01 (14336) of the large
// form's time. The limit lies below where the forms meet on even groups (64 rows a
// group, where it gives away 3 to 4%) because uneven ones meet earlier: 40 and 64 rows
// on average 328 and 348 against 331 and 335, and over 16 x [4096, 14336] 312 to 328 and
// 299 to 316 against 306 to 309 and 311 to 321. Over a grid of 638 sizes, even and uneven, the
// choice takes 2% (int8 1%) more than the better one's. (That compares the two forms;
// just past the limit of tiles the large one fills half of the GPU: 2560 rows of
// [1024, 4096] 23 us, which the tensor cores could do in 11.)
// int8: the conversion makes a tile of 64 tokens dear, and the large form shares it
// over 256 channels. 64 x [4096, 4096], bf16 results, with 24, 40, 64 (uneven) and 80
// rows each 175, 191, 276 and 381 us against 233, 232, 241 and 240; one wave without a split, K 4096:
// 0.72 of the large form's time with 12 rows a group, 0.94 with 24, 1.15 with 32, 1.36
// with 40; with a split 0.4 to 0.9.
inline bool few_rows(int E, int64_t R, int64_t M, bool i8) {
  const int64_t groups = R < E ? R : E, tiles = token_tiles(E, R, 64) * ((M + 127) / 128);
  if (i8) return tiles <= num_sms() || R <= (tiles <= 2 * num_sms() ? 24 : 48) * groups;
  return tiles <= 2 * num_sms() || R <= (tiles <= 6 * num_sms() ? 40 : 32) * groups;
}

}  // namespace mgq
