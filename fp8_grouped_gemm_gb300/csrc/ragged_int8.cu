// int8 products grouped by expert over ragged groups (offsets null: a plain
// matrix product), and the quantiser that makes their codes.
//
//   Y[r, n] = sx[r] sw[e, n] sum_k Xq[r, k] Wq[e, n, k],   r in [offsets[e], offsets[e+1])
//   s = amax / 127,  q = round(127 x / amax), a half to the even neighbour, per row
//
// GB300's tensor cores have no int8 form worth using. Every int8 value is an f16
// value, though, products of two are exact in f32, and a sum of them is exact
// while it stays below 2^24 (kPartHalves: what becomes of longer ones). So the codes
// travel as bytes, half of what bf16 would read, and become f16 beside the tensor
// cores. The tiles are those of the bf16 products: two SMs share 256 output channels
// by up to 256 tokens.
//   warp 0        TMA: 128 channels and up to 128 tokens of 128 bytes a stage
//   warps 4-11    channels: bytes -> f16 -> tensor memory, the MMA's A operand
//   warps 12-19   tokens: bytes -> f16 -> shared memory, swizzled, the B operand
//   warp 1        (CTA 0) issues the MMAs of both SMs
//   warps 20-27   epilogue: scales, full runs of 32 tokens to the TMA's stores
// The channels' operand in tensor memory leaves shared memory's bandwidth to the
// tokens' one; its stages take the columns of a second accumulator, so a tile's
// MMAs wait for the tile before to be read.
//
// Bound by the tensor cores at their f16 rate (active 87% of the time at 8192 rows
// of 4 x [8192, 4096]), short contractions by the wait between tiles, long calls by
// the power cap; float32 results of long contractions by the conversion (kPartHalves:
// tensor cores 71%, issue slots 65%). Measured: 8192^3 539-580 us (1900-2040 TFLOP/s),
// float32 668; 32768 rows over 8 x [4096, 14336] 1890, float32 2140.
#include "ragged.cuh"
#include "ragged_int8.cuh"

namespace mgq {
namespace {

constexpr int kRaw = 4, kConv = 4;                 // stages of bytes, and half stages of f16
constexpr uint32_t kRawBytes = 128 * 128;          // one operand's bytes of a stage
constexpr uint32_t kF16Bytes = 128 * 128;          // the tokens' f16 of half a stage, 64 elements
constexpr uint32_t kAcols = 32;                    // tensor memory: columns of one of the channels' half stages
constexpr int kThreads8 = 28 * 32;
// A sum of 1024 products is exact in float32 whatever the codes (128 * 128 * 1024 =
// 2^24); beyond 2^24 the tensor cores cut bits off at every step, always towards
// zero. So for float32 results of longer contractions (PARTS) the sum moves to
// registers of the epilogue every 1024 elements and is added there with rounding.
// Those registers hold 192 tokens of a tile, not 256, which leaves the tensor memory
// room for two accumulators. It costs conversions (8192^3 587 -> 675 us, 32768 rows
// over 8 x [4096, 14336] 1975 -> 2300, 1003 rows of [16384, 5120] 107 -> 130), and
// bf16 results go without: what they lose is far below their own rounding.
constexpr int kPartHalves = 1024 / 64;
__host__ __device__ constexpr int tokens_of(bool parts) { return parts ? 192 : 256; }
__host__ __device__ constexpr uint32_t acol_of(bool parts) { return parts ? 384u : 256u; }
// Registers a thread of the three kinds of warps, out of what the block is launched
// with: an epilogue warp holds 32 scaled values (96 sums) beside its addresses.
constexpr int kRegLow = 40, kRegLaunch = 72;
__host__ __device__ constexpr int reg_conv(bool parts) { return parts ? 48 : 64; }
__host__ __device__ constexpr int reg_epi(bool parts) { return parts ? 136 : 104; }
static_assert(128 * kRegLow + 512 * reg_conv(true) + 256 * reg_epi(true) <= kThreads8 * kRegLaunch, "register split");
static_assert(128 * kRegLow + 512 * reg_conv(false) + 256 * reg_epi(false) <= kThreads8 * kRegLaunch, "register split");
constexpr size_t kSmem8 = 1024 + kRaw * 2 * (size_t)kRawBytes + kConv * (size_t)kF16Bytes + 8 * (512 + kTokSlot) + 256 +
                          2 * (kMaxE + 8) * 4;
static_assert(kSmem8 <= 232448 && acol_of(true) + kConv * kAcols <= 512 && 2 * tokens_of(true) <= acol_of(true),
              "shared and tensor memory");

template <bool F32, bool PARTS>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads8, 1)
    ragged_int8_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                       const __grid_constant__ CUtensorMap tmS, const __grid_constant__ CUtensorMap tmO,
                       const RaggedArgs p) {
  constexpr int TOK = tokens_of(PARTS), NACC = PARTS ? 2 : 1;
  constexpr uint32_t kAcol = acol_of(PARTS);
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = ptx::smem_u32(smem_raw);
  uint8_t* sA = smem_raw + (((raw + 1023u) & ~1023u) - raw);   // [kRaw] bytes of the channels
  uint8_t* sB = sA + kRaw * kRawBytes;                         // [kRaw] bytes of the tokens
  uint8_t* sF = sB + kRaw * kRawBytes;                         // [kConv] f16 of the tokens
  uint8_t* sOut = sF + kConv * kF16Bytes;                      // [8 warps] store staging
  float* sX = reinterpret_cast<float*>(sOut + 8 * kTokSlot);   // [8 warps][128] token scales
  uint64_t* raw_full = reinterpret_cast<uint64_t*>(sX + 8 * 128);
  uint64_t* raw_empty = raw_full + kRaw;
  uint64_t* conv_full = raw_empty + kRaw;
  uint64_t* conv_empty = conv_full + kConv;
  uint64_t* acc_full = conv_empty + kConv;                     // [NACC]
  uint64_t* acc_empty = acc_full + NACC;
  uint64_t* drained = acc_empty + NACC;
  uint32_t* s_tmem = reinterpret_cast<uint32_t*>(drained + 1);
  volatile int* s_abort = reinterpret_cast<volatile int*>(s_tmem + 1);
  int* s_bad = reinterpret_cast<int*>(s_tmem + 2);
  volatile int* s_n = reinterpret_cast<volatile int*>(s_tmem + 3);   // [kRaw] tokens of a stage's tile, -1 after the last one
  int32_t* s_off = reinterpret_cast<int32_t*>(raw_full + 32);
  int32_t* s_cum = s_off + (kMaxE + 8);

  const int warp = __shfl_sync(0xFFFFFFFFu, (int)(threadIdx.x >> 5), 0);   // (known to be uniform)
  const uint32_t lane = threadIdx.x & 31;
  const uint32_t rank = ptx::cluster_ctarank();
  const bool leader = rank == 0;
  const int64_t pair = blockIdx.x >> 1, npairs = gridDim.x >> 1;

  if (threadIdx.x == 0) {
    for (int s = 0; s < kRaw; ++s) {
      ptx::mbar_init(&raw_full[s], 1);
      ptx::mbar_init(&raw_empty[s], 16);           // one arrival per converting warp
    }
    for (int s = 0; s < kConv; ++s) {
      ptx::mbar_init(&conv_full[s], 2 * 8);        // half of them, of both CTAs
      ptx::mbar_init(&conv_empty[s], 1);
    }
    for (int a = 0; a < NACC; ++a) {
      ptx::mbar_init(&acc_full[a], 1);
      ptx::mbar_init(&acc_empty[a], 2 * 8);        // one arrival per epilogue warp of each CTA
    }
    ptx::mbar_init(drained, 1);
    *s_abort = 0;
    ptx::fence_mbar_init();
    ptx::prefetch_tmap(&tmA);
    ptx::prefetch_tmap(&tmB);
    ptx::prefetch_tmap(&tmS);
    ptx::prefetch_tmap(&tmO);
  }
  if (warp == 1) {
    ptx::tmem_alloc_pair(s_tmem, 512);
    ptx::tmem_relinquish_pair();
  }
  ptx::grid_wait();                    // from here on: what the launch before wrote
  ptx::grid_launch();
  if (warp == 2) {
    const bool ok = load_groups<TOK>(p, s_off, s_cum, lane);
    if (lane == 0) {
      *s_bad = ok ? 0 : 1;
      if (!ok) report(p.err, MGQ_ERR_INVALID_ARG);
    }
  }
  __syncthreads();
  ptx::tc_fence_before();
  ptx::cluster_sync();
  ptx::tc_fence_after();
  const uint32_t tmem = *s_tmem;
  const bool run = *s_bad == 0;
  auto timed_out = [&]() {
    report(p.err, MGQ_ERR_TIMEOUT);
    *s_abort = 1;
  };

  if (warp < 4) ptx::setmaxnreg_dec<kRegLow>();
  if (run && warp == 0 && !p.stall && ptx::elect_one()) {
    // ------------------------------------------------------------ producer (both CTAs)
    int ecur = 0;
    uint32_t it = 0, st = 0, ph = 0;
    RaggedTile tl;
    for (int64_t t = pair; !*s_abort && ragged_tile<kFwd, TOK>(s_off, s_cum, p, t, ecur, tl); t += npairs) {
      const int half = (tl.n + 31) / 32 * 16;      // this CTA's tokens
      const int boxes = half == 128 ? 0 : (half + (int)kSmallBox - 1) / (int)kSmallBox;
      const uint32_t bytes = kRawBytes + (boxes ? boxes * kSmallBox * 128 : kRawBytes);
      for (int s = 0; s < tl.nst; ++s, ++it) {
        if (*s_abort) break;
        if (!ptx::mbar_wait(&raw_empty[st], ph ^ 1, p.wait_ns)) {
          timed_out();
          break;
        }
        s_n[st] = tl.n;
        ptx::mbar_arrive_expect_tx(&raw_full[st], bytes);
        const int32_t kx = s * kBK8, r = tl.row0 + half * (int)rank;
        ptx::tma_load_3d(sA + st * kRawBytes, &tmA, &raw_full[st], kx, (int32_t)(tl.m0 + 128 * rank), tl.e);
        if (!boxes) ptx::tma_load_3d(sB + st * kRawBytes, &tmB, &raw_full[st], kx, r, 0);
        for (int i = 0; i < boxes; ++i)
          ptx::tma_load_3d(sB + st * kRawBytes + i * kSmallBox * 128, &tmS, &raw_full[st], kx, r + i * (int)kSmallBox, 0);
        if (++st == kRaw) st = 0, ph ^= 1;
      }
    }
    if (!*s_abort && ptx::mbar_wait(&raw_empty[st], ph ^ 1, p.wait_ns)) {
      s_n[st] = -1;
      ptx::mbar_arrive(&raw_full[st]);
    }
    // after a wait that ran out: no copy may still be on its way when the CTA leaves
    if (*s_abort)
      for (uint32_t i = it > kRaw ? it - kRaw : 0; i < it; ++i)
        ptx::mbar_wait(&raw_full[i % kRaw], (i / kRaw) & 1, p.wait_ns);
  } else if (run && leader && warp == 1 && ptx::elect_one()) {
    // ------------------------------------------------------------ MMA issuer (CTA 0)
    int ecur = 0;
    uint32_t st = 0, ph = 0, tc = 0;
    RaggedTile tl;
    const uint32_t sF0 = ptx::smem_u32(sF);
    bool ok = true;
    for (int64_t t = pair; ok && ragged_tile<kFwd, TOK>(s_off, s_cum, p, t, ecur, tl); t += npairs) {
      const uint32_t idesc = ptx::idesc_f16(0, 256, (uint32_t)(tl.n + 31) / 32 * 32);
      // an accumulator a part (one loop over all half stages with a question for the
      // part's ends in it: 64 x [4096, 4096] of 80 rows, bf16, 242 -> 255 us)
      for (int s0 = 0, s1; ok && s0 < 2 * tl.nst; s0 = s1, ++tc) {
        s1 = PARTS ? min(s0 + kPartHalves, 2 * tl.nst) : 2 * tl.nst;
        const uint32_t acc = tmem + tc % NACC * TOK;
        ok = !*s_abort && ptx::mbar_wait(&acc_empty[tc % NACC], ((tc / NACC) & 1) ^ 1, p.wait_ns);
        for (int s = s0; ok && s < s1; ++s) {
          ok = !*s_abort && ptx::mbar_wait(&conv_full[st], ph, p.wait_ns);
          if (!ok) break;
          ptx::tc_fence_after();
#pragma unroll
          for (int kk = 0; kk < 4; ++kk)
            ptx::mma_f16_ta_pair(acc, tmem + kAcol + st * kAcols + kk * 8,
                                 ptx::sdesc_kmajor_sw128(sF0 + st * kF16Bytes) + kk * 2, idesc,
                                 (s > s0 || kk > 0) ? 1u : 0u);
          ptx::mma_commit_pair(&conv_empty[st], 0x3);
          if (++st == kConv) st = 0, ph ^= 1;
        }
        if (ok) ptx::mma_commit_pair(&acc_full[tc % NACC], 0x3);
      }
    }
    if (!ok) {
      timed_out();
      ptx::mma_commit_pair(drained, 0x1);          // the MMAs issued so far finish before the CTA leaves
      ptx::mbar_wait(drained, 0, p.wait_ns);
    }
  } else if (warp >= 4 && warp < 20) {
    ptx::setmaxnreg_dec<reg_conv(PARTS)>();
    // ------------------------------------------------------------ bytes to f16
    // (8 warps an operand: 32 rows each, 4 warps for each half of a stage)
    const bool chan = warp < 12;
    const uint32_t quad = warp & 3;                                     // channels: the warp's own lanes of tensor memory
    const int h = ((warp - 4) >> 2) & 1;
    const uint32_t row = quad * 32 + lane;
    uint32_t rs = 0, rph = 0, cs = h, cph = 0;                          // every second half stage
    // (a chain of latencies, which bounds tiles of few tokens: one vote and one
    // barrier of the warp a round, the codes on their way during the second wait)
    const uint32_t full0 = ptx::mapa_shared(ptx::smem_u32(conv_full), 0);
    bool ok = run;
    while (ok) {
      ok = ptx::mbar_wait(&raw_full[rs], rph, p.wait_ns);
      const int n = s_n[rs];
      uint4 c[4];
      load_codes((chan ? sA : sB) + rs * kRawBytes, row, h, c);
      ok = ok && (n < 0 || ptx::mbar_wait(&conv_empty[cs], cph ^ 1, p.wait_ns));
      ok = __all_sync(0xFFFFFFFFu, ok && !*s_abort);
      if (!ok || n < 0) break;                                          // (n < 0: no more tiles)
      if (chan) {
        ptx::tc_fence_after();
        if (PARTS) codes_to_tmem_halves(c, tmem + kAcol + cs * kAcols + ((32u * quad) << 16));
        else codes_to_tmem(c, tmem + kAcol + cs * kAcols + ((32u * quad) << 16));
        ptx::tmem_st_wait();
        ptx::tc_fence_before();
      } else if ((int)(quad * 32) < (n + 31) / 32 * 16) {               // the rows an MMA reads
        codes_to_smem(c, sF + cs * kF16Bytes, row);
        ptx::fence_proxy_async_smem();
      }
      __syncwarp();
      if (lane == 0) {
        ptx::mbar_arrive(&raw_empty[rs]);                               // (the codes are used, not only asked for)
        ptx::mbar_arrive_pair(full0 + cs * 8);
      }
      if (++rs == kRaw) rs = 0, rph ^= 1;
      if ((cs += 2) >= kConv) cs -= kConv, cph ^= 1;
    }
    if (run && !ok) timed_out();
  } else if (warp >= 20) {
    ptx::setmaxnreg_inc<reg_epi(PARTS)>();
    // ------------------------------------------------------------ epilogue (both CTAs)
    const uint32_t q = warp & 3;
    const uint32_t half = (uint32_t)(warp - 20) >> 2;
    const uint32_t empty0 = ptx::mapa_shared(ptx::smem_u32(acc_empty), 0);
    float* sx = sX + (warp - 20) * 128;
    uint8_t* slot = sOut + (warp - 20) * kTokSlot;
    int ecur = 0;
    uint32_t tc = 0;
    RaggedTile tl;
    // the next accumulator, and its release once it is read
    auto wait_acc = [&]() {
      bool got = *s_abort == 0;
      got = got && ptx::mbar_wait(&acc_full[tc % NACC], (tc / NACC) & 1, p.wait_ns);
      if (!__all_sync(0xFFFFFFFFu, got)) {
        timed_out();
        return false;
      }
      ptx::tc_fence_after();
      return true;
    };
    auto release_acc = [&]() {
      ptx::tc_fence_before();
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive_pair(empty0 + tc % NACC * 8);
      ++tc;
    };
    for (int64_t t = pair; run && ragged_tile<kFwd, TOK>(s_off, s_cum, p, t, ecur, tl); t += npairs) {
      const int64_t m0 = tl.m0 + (int)(128 * rank + 32 * q);
      const float sw = m0 + lane < p.M ? p.sw[tl.e * p.M + m0 + lane] : 0.0f;
      __syncwarp();
#pragma unroll
      for (int i = 0; i < TOK / 64; ++i) {         // runs of 32 tokens, every second run
        const int c = 32 * (int)half + 64 * i + (int)lane;
        sx[32 * i + lane] = c < tl.n ? p.sx[(int64_t)tl.row0 + c] : 0.0f;
      }
      __syncwarp();
      auto scale_and_store = [&](int i, float (&v)[32]) {
        const int c = 32 * (int)half + 64 * i;
#pragma unroll
        for (int j = 0; j < 32; j += 4) {
          const float4 x = *reinterpret_cast<const float4*>(sx + 32 * i + j);
          v[j] *= x.x * sw;
          v[j + 1] *= x.y * sw;
          v[j + 2] *= x.z * sw;
          v[j + 3] *= x.w * sw;
        }
        if (tl.n - c >= 32 && m0 < p.M) send_tokens<F32>(&tmO, slot, v, tl.row0 + c, (int32_t)m0, lane);
        else store_tokens<F32>(p.out, p.ldo, v, (int64_t)tl.row0 + c, tl.n - c, m0, p.M, lane);
      };
      auto load = [&](int i, float (&v)[32], bool add) {
#pragma unroll
        for (int h = 0; h < 32; h += 16) {
          uint32_t r[16];
          ptx::tmem_ld_32x32b_x16(tmem + tc % NACC * TOK + 32 * half + 64 * i + h + ((q * 32) << 16), r);
          ptx::tmem_ld_wait();
#pragma unroll
          for (int j = 0; j < 16; ++j) v[h + j] = add ? v[h + j] + __uint_as_float(r[j]) : __uint_as_float(r[j]);
        }
      };
      if (PARTS) {
        float v[TOK / 64][32];
        bool got = true;
        const int parts = (2 * tl.nst + kPartHalves - 1) / kPartHalves;
        for (int part = 0; part < parts; ++part) {
          if (!(got = wait_acc())) break;
#pragma unroll
          for (int i = 0; i < TOK / 64; ++i)
            if (32 * (int)half + 64 * i < tl.n) load(i, v[i], part > 0);
          release_acc();
        }
        if (!got) break;
#pragma unroll
        for (int i = 0; i < TOK / 64; ++i)
          if (32 * (int)half + 64 * i < tl.n) scale_and_store(i, v[i]);
      } else {
        if (!wait_acc()) break;
        for (int i = 0; 32 * (int)half + 64 * i < tl.n; ++i) {
          float v[32];
          load(i, v, false);
          if (32 * (int)half + 64 * (i + 1) >= tl.n) release_acc();   // it is read: the next tile may begin
          scale_and_store(i, v);
        }
        if (32 * (int)half >= tl.n) release_acc(); // (no tokens for this warp)
      }
    }
    if (lane == 0) ptx::bulk_wait0();              // this warp's stores are complete
  }
  __syncthreads();
  ptx::tc_fence_before();
  ptx::cluster_sync();                 // the peer's MMAs and reads are finished before freeing
  ptx::tc_fence_after();
  if (warp == 1) {
    __syncwarp();
    ptx::tmem_dealloc_pair(tmem, 512);
  }
}

template <bool F32, bool PARTS>
int launch_int8(const CUtensorMap& ta, const CUtensorMap& tb, const CUtensorMap& ts, const CUtensorMap& to,
                const RaggedArgs& p, int64_t max_tiles, cudaStream_t s) {
  auto kern = ragged_int8_kernel<F32, PARTS>;
  static OncePerDevice once;
  if (!once.run([&](int) {
        // (a build that launches with fewer registers could not serve the split)
        cudaFuncAttributes at;
        return cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSmem8) == cudaSuccess &&
               cudaFuncGetAttributes(&at, kern) == cudaSuccess && at.numRegs >= kRegLaunch;
      }))
    return MGQ_ERR_CUDA;
  const int64_t pairs = min((int64_t)(num_sms() / 2), max_tiles);
  return launch_after(kern, dim3((unsigned)(2 * max(pairs, (int64_t)1))), kThreads8, kSmem8, 1, s, ta, tb, ts, to, p)
             ? MGQ_OK
             : MGQ_ERR_CUDA;
}

// ---------------------------------------------------------------------------
// Row quantiser, bound by memory: 16384 x 4096 in 30.7 us (6.6 TB/s), one row of 4096
// in 1.4. G threads a row, each up to two units of 16 elements in
// registers (longer rows are read twice). The code is round(127 x / amax) of the
// exact quotient, decided in float32: with x = a 2^i, amax = b 2^j (8-bit a, b) a
// quotient that is not halfway between two integers is away from it by at least
// 1 / (254 * 255) = 2^-16 of its value, and one that is has 9 significant bits; so
// the product with the rounded 127 / amax (within 2^-22) is rounded to 20 bits
// first, which puts the halves back in place and moves nothing across one.

struct Quant8Args {
  const uint16_t* x;
  int64_t ldx, T;
  int K;
  int8_t* codes;
  float* scale;
};

__device__ __forceinline__ uint32_t code8(float x, float pre, float inv) {
  const uint32_t b = __float_as_uint(__fmul_rn(__fmul_rn(x, pre), inv));
  return __float_as_uint(__fadd_rn(__uint_as_float((b + 8u) & ~15u), 12582912.0f));    // 1.5 2^23: integer in the low bits
}
__device__ __forceinline__ uint32_t codes4(uint32_t w0, uint32_t w1, float pre, float inv) {
  const uint32_t a = __byte_perm(code8(bf16_lo(w0), pre, inv), code8(bf16_hi(w0), pre, inv), 0x0040);
  const uint32_t b = __byte_perm(code8(bf16_lo(w1), pre, inv), code8(bf16_hi(w1), pre, inv), 0x0040);
  return __byte_perm(a, b, 0x5410);
}

template <int G>
__global__ void __launch_bounds__(G < 128 ? 128 : G) rows_quant8_kernel(Quant8Args a) {
  constexpr int kRows = G < 128 ? 128 / G : 1;
  __shared__ uint32_t s_max[G / 32];
  const int tid = threadIdx.x % G, lane = threadIdx.x & 31;
  const int64_t row = blockIdx.x * (int64_t)kRows + threadIdx.x / G;
  if (row >= a.T) return;                          // (whole warps; a row of several warps is the CTA)
  ptx::grid_wait();
  ptx::grid_launch();
  const uint4* x = reinterpret_cast<const uint4*>(a.x + row * a.ldx);
  const int units = a.K / 16;
  uint4 w[2][2];
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int u = tid + i * G;
    if (u < units) {
      w[i][0] = x[2 * u];
      w[i][1] = x[2 * u + 1];
    } else {
      w[i][0] = w[i][1] = make_uint4(0, 0, 0, 0);
    }
  }
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      m = absmax_bf16x2(m, w[i][h].x);
      m = absmax_bf16x2(m, w[i][h].y);
      m = absmax_bf16x2(m, w[i][h].z);
      m = absmax_bf16x2(m, w[i][h].w);
    }
  for (int u = tid + 2 * G; u < units; u += G)
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const uint4 v = x[2 * u + h];
      m = absmax_bf16x2(absmax_bf16x2(absmax_bf16x2(absmax_bf16x2(m, v.x), v.y), v.z), v.w);
    }
  uint32_t bits = fold_bf16x2(m);
  bits = __reduce_max_sync(0xFFFFFFFFu, bits);
  if (G > 32) {
    if (lane == 0) s_max[threadIdx.x >> 5] = bits;
    __syncthreads();
    bits = lane < G / 32 ? s_max[lane] : 0u;
    bits = __reduce_max_sync(0xFFFFFFFFu, bits);
  }
  const bool finite = bits < 0x7F800000u;
  const float amax = __uint_as_float(bits);
  // (127 / amax overflows below 2^-121: such rows are scaled up first, exactly)
  const float pre = amax < 0x1p-100f ? 0x1p100f : 1.0f;
  const float inv = !finite || amax == 0.0f ? 0.0f : __fdiv_rn(127.0f, __fmul_rn(amax, pre));
  if (tid == 0) a.scale[row] = finite ? __fdiv_rn(amax, 127.0f) : __uint_as_float(0x7FC00000u);
  uint4* out = reinterpret_cast<uint4*>(a.codes + row * a.K);
  auto put = [&](int u, const uint4& p, const uint4& q) {
    out[u] = finite ? make_uint4(codes4(p.x, p.y, pre, inv), codes4(p.z, p.w, pre, inv), codes4(q.x, q.y, pre, inv),
                                 codes4(q.z, q.w, pre, inv))
                    : make_uint4(0, 0, 0, 0);
  };
#pragma unroll
  for (int i = 0; i < 2; ++i)
    if (tid + i * G < units) put(tid + i * G, w[i][0], w[i][1]);
  for (int u = tid + 2 * G; u < units; u += G) put(u, x[2 * u], x[2 * u + 1]);
}

}  // namespace
}  // namespace mgq

using namespace mgq;

extern "C" {

int mgq_ragged_gemm_int8(const int8_t* x, int64_t ldx, const float* x_scale, const int8_t* w, const float* w_scale,
                         const int32_t* offsets, int E, int64_t R, int64_t N, int64_t K, void* y, int64_t ldy,
                         int out_dtype, void* stream) {
  MGQ_CHECK_ARG(E >= 1 && E <= kMaxE && R >= 0 && R < (1ll << 31) - 512 && N > 0 && K > 0);
  MGQ_CHECK_ARG(N % 8 == 0 && K % 16 == 0 && N < (1ll << 31) - 512 && K < (1ll << 31) - 512);
  MGQ_CHECK_ARG((offsets || E == 1) && (reinterpret_cast<uintptr_t>(offsets) & 3u) == 0);
  MGQ_CHECK_ARG(out_dtype == MGQ_OUT_BF16 || out_dtype == MGQ_OUT_F32);
  MGQ_CHECK_ARG(ldx >= K && ldx % 16 == 0 && ldx < (1ll << 39) && ldy >= N && ldy % 8 == 0 && ldy < (1ll << 38));
  MGQ_CHECK_ARG(R == 0 || (x && x_scale && w && w_scale && y));
  MGQ_CHECK_ARG(aligned16(x) && aligned16(w) && aligned16(y) && (reinterpret_cast<uintptr_t>(x_scale) & 3u) == 0 &&
                aligned16(w_scale));
  if (R == 0) return MGQ_OK;
  RaggedArgs p{};
  p.err = error_word();
  if (!p.err) return MGQ_ERR_CUDA;
  p.offsets = offsets;
  p.E = E;
  p.R = R;
  p.M = N;
  p.C = K;
  p.out = y;
  p.ldo = ldy;
  p.out_f32 = out_dtype == MGQ_OUT_F32;
  p.bk = kBK8;
  p.sx = x_scale;
  p.sw = w_scale;
  debug_knobs(&p.stall, &p.wait_ns);
  const bool few = few_rows(E, R, N, true);
  CUtensorMap ta, tb, ts, to;
  if (few) {
    if (!encode_tmap_swz_3d(&ta, w, 1, {(uint64_t)K, (uint64_t)N, (uint64_t)E}, K, N * K, {128, 128, 1}) ||
        !encode_tmap_swz_3d(&ts, x, 1, {(uint64_t)K, (uint64_t)R, 1}, ldx, R * ldx, {128, kFewBox, 1}))
      return MGQ_ERR_CUDA;
    return run_few(kFwd, true, ta, ts, p, as_stream(stream));
  }
  if (!encode_tmap_swz_3d(&ta, w, 1, {(uint64_t)K, (uint64_t)N, (uint64_t)E}, K, N * K, {128, 128, 1}) ||
      !encode_tmap_swz_3d(&tb, x, 1, {(uint64_t)K, (uint64_t)R, 1}, ldx, R * ldx, {128, 128, 1}) ||
      !encode_tmap_swz_3d(&ts, x, 1, {(uint64_t)K, (uint64_t)R, 1}, ldx, R * ldx, {128, kSmallBox, 1}) ||
      !encode_out(&to, y, R, N, ldy, p.out_f32))
    return MGQ_ERR_CUDA;
  const bool parts = p.out_f32 && K > 1024;
  const int64_t tiles = token_tiles(E, R, tokens_of(parts)) * ((N + kTile - 1) / kTile);
  return parts       ? launch_int8<true, true>(ta, tb, ts, to, p, tiles, as_stream(stream))
         : p.out_f32 ? launch_int8<true, false>(ta, tb, ts, to, p, tiles, as_stream(stream))
                     : launch_int8<false, false>(ta, tb, ts, to, p, tiles, as_stream(stream));
}

int mgq_rows_quantize_int8(const void* x_bf16, int64_t ldx, int64_t T, int64_t K, int8_t* codes, float* scale,
                           void* stream) {
  MGQ_CHECK_ARG(T >= 0 && T < (1ll << 31) && K > 0 && K % 16 == 0 && K < (1ll << 31));
  MGQ_CHECK_ARG(ldx >= K && ldx % 8 == 0 && (T == 0 || (x_bf16 && codes && scale)));
  MGQ_CHECK_ARG(aligned16(x_bf16) && aligned16(codes) && (reinterpret_cast<uintptr_t>(scale) & 3u) == 0);
  if (T == 0) return MGQ_OK;
  Quant8Args a{static_cast<const uint16_t*>(x_bf16), ldx, T, (int)K, codes, scale};
  cudaStream_t s = as_stream(stream);
  const int64_t units = K / 16;
  const bool ok = units <= 64    ? launch_after(rows_quant8_kernel<32>, dim3((unsigned)((T + 3) / 4)), 128, 0, 1, s, a)
                  : units <= 256 ? launch_after(rows_quant8_kernel<128>, dim3((unsigned)T), 128, 0, 1, s, a)
                                 : launch_after(rows_quant8_kernel<512>, dim3((unsigned)T), 512, 0, 1, s, a);
  return ok ? MGQ_OK : MGQ_ERR_CUDA;
}

}  // extern "C"
