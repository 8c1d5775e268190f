// The products over ragged groups for few rows a group (decode batches, short
// micro-batches): bound by one read of the weights of the groups that have rows.
//
// One CTA a tile of 128 output channels by up to 64 tokens of one group, the
// weights on the tensor cores' M side, tokens on the N side in steps of 16. Two
// CTAs share an SM, so that one streams weights while the other starts or ends.
// Where the tiles are too few to keep the memory busy, a cluster of up to 8 CTAs
// splits the contraction; the parts meet in shared memory over the cluster and
// are added in the order of the ranks, so the result does not depend on timing.
// int8 weights become f16 on their way to tensor memory, as in the large form, and
// a CTA takes one tile after the other.
//
// Measured: 32 rows over 8 x [28672, 4096], bf16 255 us (7.4 TB/s of weights), int8
// 147 (6.4 TB/s; float32 153); one row of [4096, 4096] 6.6 and 6.8 us (float32 7.1).
#include "ragged.cuh"
#include "ragged_int8.cuh"

namespace mgq {
namespace {

constexpr int kFewTok = 64;                        // tokens of a tile at most
constexpr uint32_t kFewA = 128 * 128;              // bytes of the weights a stage
constexpr uint32_t kFewB = kFewTok * 128;          // bytes of the tokens a stage
constexpr uint32_t kFewF = kFewTok * 256;          // int8: the tokens' f16 of a stage
__host__ __device__ constexpr int few_stages(bool i8) { return i8 ? 3 : 4; }
constexpr int kFewConv = 2;                        // int8: stages of f16
__host__ __device__ constexpr int few_threads(bool i8) { return i8 ? 256 : 192; }
__host__ __device__ constexpr size_t few_smem(bool i8) {
  return 1024 + few_stages(i8) * (size_t)(kFewA + kFewB) + (i8 ? kFewConv * (size_t)kFewF : 0) + 256 + (kMaxE + 8) * 4;
}
static_assert(2 * (few_smem(true) + 1024) <= 233472 && 2 * (few_smem(false) + 1024) <= 233472, "two CTAs an SM");
static_assert(few_stages(true) * (kFewA + kFewB) >= kFewTok * 128 * 4, "room for a partial result");
// tensor memory: two accumulators, for int8 with the weights' f16 between them
constexpr uint32_t kFewAcol = 64, kFewCols8 = 256, kFewCols = 128;
template <bool I8>
constexpr uint32_t kFewAcc2 = I8 ? kFewAcol + kFewConv * 64 : 64;
static_assert(kFewAcc2<true> + 64 <= kFewCols8, "tensor memory");
// Stages after which a float32 result's sum moves to registers, where it is added with
// rounding: 512 elements of bf16 as in the large form; int8: 1024, whose sum is exact
// whatever the codes (128 * 128 * 1024 = 2^24; beyond that the tensor cores cut off).
// (int8 without it: 32 rows over 8 x [28672, 4096], float32 148 us against 153.)
constexpr int kFewPromote = 8;

struct FewTile {
  int e, row0, n;
  int64_t m0;
};

// A warp's view of the groups, for the search: each lane has the token tiles of its
// run of groups, and the sum of those up to and with its own.
struct FewGroups {
  uint32_t mine, inc, nM;
  int per;
};

// s_off holds the offsets; a whole warp. False for offsets that are no row partition.
__device__ __forceinline__ bool few_groups(const RaggedArgs& p, const int32_t* s_off, uint32_t lane, FewGroups& g) {
  g.per = (p.E + 31) / 32;
  g.nM = (uint32_t)((p.M + 127) / 128);
  const int e0 = min((int)lane * g.per, p.E), e1 = min(e0 + g.per, p.E);
  uint32_t mine = 0;
  bool ok = true;
  for (int e = e0, lo = s_off[e0]; e < e1; ++e) {
    const int hi = s_off[e + 1];
    ok &= lo >= 0 && lo <= hi && hi <= p.R;
    mine += (uint32_t)(max(hi - lo, 0) + kFewTok - 1) / kFewTok;
    lo = hi;
  }
  uint32_t inc = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t v = __shfl_up_sync(0xFFFFFFFFu, inc, o);
    if (lane >= (uint32_t)o) inc += v;
  }
  g.mine = mine;
  g.inc = inc;
  return __all_sync(0xFFFFFFFFu, ok);
}

// Tile t: groups in order, a group's channel tiles, its token tiles fastest (they
// share the weights). A whole warp. False if there is no such tile. (Tile numbers
// are below 2^31: the launch sees to it.)
__device__ __forceinline__ bool few_tile(const FewGroups& g, const int32_t* s_off, uint32_t t, FewTile& tl) {
  const uint32_t at = __ballot_sync(0xFFFFFFFFu, g.inc * g.nM > t);
  if (!at) return false;
  const int src = __ffs(at) - 1;
  // every lane walks that lane's groups
  uint32_t local = t - __shfl_sync(0xFFFFFFFFu, g.inc - g.mine, src) * g.nM, tiles = 1;
  int e = src * g.per, lo = s_off[e];
  for (;; ++e) {
    const int hi = s_off[e + 1];
    tiles = (uint32_t)(hi - lo + kFewTok - 1) / kFewTok;
    if (local < tiles * g.nM) break;
    local -= tiles * g.nM;
    lo = hi;
  }
  const uint32_t m = local / tiles;
  tl.e = e;
  tl.row0 = lo + (int)(local - m * tiles) * kFewTok;
  tl.n = min(kFewTok, s_off[e + 1] - tl.row0);
  tl.m0 = (int64_t)m * 128;
  return true;
}

__device__ __forceinline__ float4 ld_cluster_f32x4(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(addr)
               : "memory");
  return v;
}

template <int OP, bool I8, bool F32>
__global__ void __launch_bounds__(few_threads(I8), 2)
    ragged_few_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                      const RaggedArgs p, int split) {
  constexpr int ST = few_stages(I8);
  constexpr bool kAmn = OP == kDgrad;
  constexpr bool kParts = F32;
  constexpr int kElems = I8 ? kBK8 : 64;           // of the contraction a stage
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = ptx::smem_u32(smem_raw);
  uint8_t* sA = smem_raw + (((raw + 1023u) & ~1023u) - raw);
  uint8_t* sB = sA + ST * kFewA;
  uint8_t* sF = sB + ST * kFewB;
  uint64_t* full = reinterpret_cast<uint64_t*>(sF + (I8 ? kFewConv * kFewF : 0));
  uint64_t* empty = full + ST;
  uint64_t* conv_full = empty + ST;                // [kFewConv]
  uint64_t* conv_empty = conv_full + kFewConv;
  uint64_t* acc_full = conv_empty + kFewConv;      // [2]
  uint64_t* acc_empty = acc_full + 2;              // [2]
  uint64_t* drained = acc_empty + 2;
  uint32_t* s_tmem = reinterpret_cast<uint32_t*>(drained + 1);
  volatile int* s_abort = reinterpret_cast<volatile int*>(s_tmem + 1);
  int32_t* s_off = reinterpret_cast<int32_t*>(full + 32);

  const int warp = __shfl_sync(0xFFFFFFFFu, (int)(threadIdx.x >> 5), 0);   // (known to be uniform)
  const uint32_t lane = threadIdx.x & 31;
  const int rank = split > 1 ? (int)ptx::cluster_ctarank() : 0;

  if (threadIdx.x == 0) {
    for (int s = 0; s < ST; ++s) {
      ptx::mbar_init(&full[s], 1);
      ptx::mbar_init(&empty[s], I8 ? 6 : 1);       // int8: one arrival per converting warp
    }
    for (int s = 0; s < kFewConv; ++s) {
      ptx::mbar_init(&conv_full[s], 6);
      ptx::mbar_init(&conv_empty[s], 1);
    }
    for (int a = 0; a < 2; ++a) {
      ptx::mbar_init(&acc_full[a], 1);
      ptx::mbar_init(&acc_empty[a], 4);            // one arrival per epilogue warp
    }
    ptx::mbar_init(drained, 1);
    *s_abort = 0;
    ptx::fence_mbar_init();
    ptx::prefetch_tmap(&tmA);
    ptx::prefetch_tmap(&tmB);
  }
  if (warp == 1) {
    ptx::tmem_alloc(s_tmem, I8 ? kFewCols8 : kFewCols);
    ptx::tmem_relinquish();
  }
  ptx::grid_wait();                                // from here on: what the launch before wrote
  ptx::grid_launch();
  for (int i = threadIdx.x; i <= p.E; i += few_threads(I8)) s_off[i] = p.offsets ? p.offsets[i] : i ? (int)p.R : 0;
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  const uint32_t tmem = *s_tmem;
  FewGroups groups;
  const bool part = few_groups(p, s_off, lane, groups);
  if (!part && blockIdx.x == 0 && threadIdx.x == 0) report(p.err, MGQ_ERR_INVALID_ARG);
  // the first tile; int8 without a split takes every gridDim.x-th after it
  FewTile tl{0, 0, 1, 0};
  uint32_t tile = blockIdx.x / split;
  const bool run = part && few_tile(groups, s_off, tile, tl);
  auto next_tile = [&]() { return I8 && split == 1 && few_tile(groups, s_off, tile += gridDim.x, tl); };
  // this rank's stages of the contraction
  const int nst = (int)((p.C + kElems - 1) / kElems), chunk = (nst + split - 1) / split;
  const int s0 = min(nst, rank * chunk), ns = min(nst, s0 + chunk) - s0;
  auto timed_out = [&]() {
    report(p.err, MGQ_ERR_TIMEOUT);
    *s_abort = 1;
  };

  if (run && warp == 0 && !p.stall && (I8 || ptx::elect_one())) {
    // ------------------------------------------------------------ producer
    // (int8: the whole warp, which looks for the next tile together; bf16 has one tile, and
    // the elected lane alone is 0.05 to 0.1 us faster. The same in the next warp.)
    uint32_t it = 0, st = 0, ph = 0;               // (of the electing lane, the same one throughout)
    const bool me = !I8 || ptx::elect_one();
    do {
      const int boxes = (tl.n + kFewBox - 1) / kFewBox;
      for (int i = 0; me && i < ns; ++i, ++it) {
        if (*s_abort) break;
        if (!ptx::mbar_wait(&empty[st], ph ^ 1, p.wait_ns)) {
          timed_out();
          break;
        }
        ptx::mbar_arrive_expect_tx(&full[st], kFewA + boxes * kFewBox * 128);
        const int32_t kx = (s0 + i) * kElems;
        if (kAmn) {                                // two chunks of 64 channels
          ptx::tma_load_3d(sA + st * kFewA, &tmA, &full[st], (int32_t)tl.m0, kx, tl.e);
          ptx::tma_load_3d(sA + st * kFewA + kFewA / 2, &tmA, &full[st], (int32_t)tl.m0 + 64, kx, tl.e);
        } else {
          ptx::tma_load_3d(sA + st * kFewA, &tmA, &full[st], kx, (int32_t)tl.m0, tl.e);
        }
        for (int b = 0; b < boxes; ++b)
          ptx::tma_load_3d(sB + st * kFewB + b * kFewBox * 128, &tmB, &full[st], kx, tl.row0 + b * kFewBox, 0);
        if (++st == ST) st = 0, ph ^= 1;
      }
      if (I8) __syncwarp();
    } while (I8 && !__any_sync(0xFFFFFFFFu, *s_abort != 0) && next_tile());
    if (me && *s_abort)                            // no copy may be on its way when the CTA leaves
      for (uint32_t j = it > ST ? it - ST : 0; j < it; ++j) ptx::mbar_wait(&full[j % ST], (j / ST) & 1, p.wait_ns);
    if (I8) __syncwarp();
  } else if (run && warp == 1 && (I8 || ptx::elect_one())) {
    // ------------------------------------------------------------ MMA issuer
    const uint32_t sA0 = ptx::smem_u32(sA), sB0 = ptx::smem_u32(sB), sF0 = ptx::smem_u32(sF);
    uint32_t st = 0, ph = 0, pc = 0;               // stage of its operands, accumulator
    bool ok = true;
    const bool me = !I8 || ptx::elect_one();
    do {
      const uint32_t idesc = ptx::idesc_f16(I8 ? 0 : 1, 128, (uint32_t)(tl.n + kFewBox - 1) / kFewBox * kFewBox) |
                             ptx::idesc_mn_major(kAmn, false);
      for (int i = 0; me && i < ns; ++i) {
        const bool first = kParts ? i % kFewPromote == 0 : i == 0;
        const uint32_t acc = tmem + (pc & 1) * kFewAcc2<I8>;
        if ((I8 || kParts) && first) ok = ptx::mbar_wait(&acc_empty[pc & 1], ((pc >> 1) & 1) ^ 1, p.wait_ns);
        ok = ok && !*s_abort && ptx::mbar_wait(I8 ? &conv_full[st] : &full[st], ph, p.wait_ns);
        if (!ok) break;
        ptx::tc_fence_after();
        if (I8) {
#pragma unroll
          for (int kk = 0; kk < 8; ++kk)
            ptx::mma_f16_ta(acc, tmem + kFewAcol + st * 64 + kk * 8,
                            ptx::sdesc_kmajor_sw128(sF0 + st * kFewF + (kk >> 2) * (kFewF / 2)) + (kk & 3) * 2, idesc,
                            (!first || kk > 0) ? 1u : 0u);
          ptx::mma_commit(&conv_empty[st]);
        } else {
          const uint64_t ad = kAmn ? ptx::sdesc_mnmajor_sw128_chunks(sA0 + st * kFewA, kFewA / 2)
                                   : ptx::sdesc_kmajor_sw128(sA0 + st * kFewA);
          const uint64_t bd = ptx::sdesc_kmajor_sw128(sB0 + st * kFewB);
#pragma unroll
          for (int kk = 0; kk < 4; ++kk)
            ptx::mma_f16(acc, ad + kk * (kAmn ? 128 : 2), bd + kk * 2, idesc, (!first || kk > 0) ? 1u : 0u);
          ptx::mma_commit(&empty[st]);
        }
        if (++st == (I8 ? kFewConv : ST)) st = 0, ph ^= 1;
        if (i == ns - 1 || (kParts && i % kFewPromote == kFewPromote - 1)) ptx::mma_commit(&acc_full[pc++ & 1]);
      }
      if (I8) __syncwarp();
    } while (I8 && __all_sync(0xFFFFFFFFu, ok) && next_tile());
    if (!ok) {                                     // (the electing lane)
      timed_out();
      ptx::mma_commit(drained);                    // the MMAs issued so far finish before the CTA leaves
      ptx::mbar_wait(drained, 0, p.wait_ns);
    }
    if (I8) __syncwarp();
  } else if (run && warp >= 2) {
    // int8: which rows this warp converts (warps 2-5 channels, 6-7 tokens)
    const bool chan = warp < 6;
    const uint32_t q = warp & 3, row = (chan ? q : warp - 6) * 32 + lane;
    uint32_t rs = 0, rph = 0, cs = 0, cph = 0, pc = 0;
    bool ok = true;
    const uint32_t lanes = tmem + ((q * 32) << 16);
    do {
      const int n = tl.n;
      float v[kParts ? kFewTok : 16];
      int parts = ns == 0 ? 0 : kParts ? (ns + kFewPromote - 1) / kFewPromote : 1;   // still to be taken
#pragma unroll
      for (int j = 0; j < (kParts ? kFewTok : 16); ++j) v[j] = 0.0f;
      auto wait_acc = [&]() {
        bool got = *s_abort == 0;
        got = got && ptx::mbar_wait(&acc_full[pc & 1], (pc >> 1) & 1, p.wait_ns);
        got = __all_sync(0xFFFFFFFFu, got);
        if (!got) timed_out();
        ptx::tc_fence_after();
        return got;
      };
      auto release_acc = [&]() {
        ptx::tc_fence_before();
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(&acc_empty[pc & 1]);
        ++pc;
      };
      auto take_part = [&]() {                     // the next accumulator's values into the sums
        if (!wait_acc()) return false;
#pragma unroll
        for (int h = 0; h < kFewTok; h += 16) {
          if (h >= n) break;
          uint32_t r[16];
          ptx::tmem_ld_32x32b_x16(lanes + (pc & 1) * kFewAcc2<I8> + h, r);
          ptx::tmem_ld_wait();
#pragma unroll
          for (int j = 0; j < 16; ++j) v[kParts ? h + j : j] += __uint_as_float(r[j]);
        }
        release_acc();
        --parts;
        return true;
      };
      if (I8) {
        // -------------------------------------------------------- bytes to f16
        const bool mine = chan || (int)(row - lane) < (n + kFewBox - 1) / kFewBox * kFewBox;
        for (int i = 0; i < ns; ++i) {
          ok = *s_abort == 0;
          ok = ok && ptx::mbar_wait(&full[rs], rph, p.wait_ns);
          // On their way during the second wait: all the codes, or half of them where the
          // registers hold sums (both halves: 32 rows over 8 x [28672, 4096] 153 -> 160 us).
          uint4 c[kParts ? 1 : 2][4];
          const uint8_t* src = chan ? sA + rs * kFewA : sB + rs * kFewB;
          if (mine) {
            load_codes(src, row, 0, c[0]);
            if (!kParts) load_codes(src, row, 1, c[kParts ? 0 : 1]);
          }
          ok = ok && ptx::mbar_wait(&conv_empty[cs], cph ^ 1, p.wait_ns);
          ok = __all_sync(0xFFFFFFFFu, ok);
          if (!ok) break;
          if (chan) {
            ptx::tc_fence_after();
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              if (kParts && h) load_codes(src, row, 1, c[0]);
              const uint32_t at = tmem + kFewAcol + cs * 64 + 32 * h + ((32u * q) << 16);
              if (kParts) codes_to_tmem_halves(c[0], at);
              else codes_to_tmem(c[kParts ? 0 : h], at);
            }
            ptx::tmem_st_wait();
            ptx::tc_fence_before();
          } else if (mine) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              if (kParts && h) load_codes(src, row, 1, c[0]);
              codes_to_smem(c[kParts ? 0 : h], sF + cs * kFewF + h * (kFewF / 2), row);
            }
            ptx::fence_proxy_async_smem();
          }
          __syncwarp();
          if (lane == 0) {
            ptx::mbar_arrive(&empty[rs]);          // (only now that the codes are used: a read of them may
            ptx::mbar_arrive(&conv_full[cs]);      // still be under way after an arrival that follows it)
          }
          if (++rs == ST) rs = 0, rph ^= 1;
          if (++cs == kFewConv) cs = 0, cph ^= 1;
          // A part is taken two stages after its last one: its MMAs have then finished
          // (this stage's place in the ring had waited for them), and the accumulator is
          // free again before it is needed.
          if (kParts && chan && i > kFewPromote && i % kFewPromote == 1 && !(ok = take_part())) break;
        }
        if (!ok) timed_out();
      }
      if (!chan || !ok) continue;
      // ---------------------------------------------------------- the result, channels as lanes
      const int64_t ch = tl.m0 + 32 * q + lane;
      const float sw = I8 && split == 1 && ch < p.M ? p.sw[tl.e * p.M + ch] : 0.0f;
      const bool summed = parts > 0;
      if (kParts) {
        while (ok && parts > 0) ok = take_part();
      } else if (parts) {
        ok = wait_acc();
      }
      if (!ok) break;
#pragma unroll
      for (int h = 0; h < kFewTok; h += 16) {
        if (h >= n) break;
        float x[16];
        if (!kParts && summed) {
          uint32_t r[16];
          ptx::tmem_ld_32x32b_x16(lanes + (pc & 1) * kFewAcc2<I8> + h, r);
          ptx::tmem_ld_wait();
#pragma unroll
          for (int j = 0; j < 16; ++j) x[j] = __uint_as_float(r[j]);
        } else {
#pragma unroll
          for (int j = 0; j < 16; ++j) x[j] = v[kParts ? h + j : j];
        }
        if (split > 1) {                           // [token][channel], for the sum at the end
          float* part_out = reinterpret_cast<float*>(sA) + q * 32 + lane;
#pragma unroll
          for (int j = 0; j < 16; ++j) part_out[(h + j) * 128] = x[j];
        } else {
          if (I8) {
            const float sx = (int)lane < min(16, n - h) ? p.sx[(int64_t)tl.row0 + h + lane] : 0.0f;
#pragma unroll
            for (int j = 0; j < 16; ++j) x[j] *= __shfl_sync(0xFFFFFFFFu, sx, j) * sw;
          }
          store_tokens<F32>(p.out, p.ldo, x, (int64_t)tl.row0 + h, n - h, tl.m0 + 32 * q, p.M, lane);
        }
      }
      if (!kParts && summed) release_acc();
    } while (ok && next_tile());
  }
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  if (warp == 1) {
    __syncwarp();
    ptx::tmem_dealloc(tmem, I8 ? kFewCols8 : kFewCols);
  }
  if (split == 1 || !run) return;                  // (the whole cluster)
  const int e = tl.e, row0 = tl.row0, n = tl.n;
  const int64_t m0 = tl.m0;
  ptx::cluster_sync();                             // every part is in place
  // tokens rank, rank + split, ..: a warp each, four channels a lane
  const int64_t ch = m0 + 4 * lane;
  const bool in = ch < p.M && !*s_abort;
  const uint32_t mine = ptx::smem_u32(sA) + lane * 16;
  float4 sw = make_float4(1.0f, 1.0f, 1.0f, 1.0f);
  if (I8 && in) sw = *reinterpret_cast<const float4*>(p.sw + e * p.M + ch);
  constexpr int kWarps = few_threads(I8) / 32;
  // (only lanes that use what they read: the last barrier does not wait for a load whose
  // value nobody needs, and the peer's shared memory may be gone after it)
  for (int j = rank + split * warp; in && j < n; j += split * kWarps) {
    float4 s = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    for (int r = 0; r < split; ++r) {
      const float4 x = ld_cluster_f32x4(ptx::mapa_shared(mine + j * 512, r));
      s.x += x.x;
      s.y += x.y;
      s.z += x.z;
      s.w += x.w;
    }
    const int64_t tok = (int64_t)row0 + j;
    if (I8) {
      const float sx = p.sx[tok];
      s.x *= sx * sw.x;
      s.y *= sx * sw.y;
      s.z *= sx * sw.z;
      s.w *= sx * sw.w;
    }
    if (F32) *reinterpret_cast<float4*>(static_cast<float*>(p.out) + tok * p.ldo + ch) = s;
    else
      *reinterpret_cast<uint2*>(static_cast<uint16_t*>(p.out) + tok * p.ldo + ch) =
          make_uint2(pack_bf16x2(s.x, s.y), pack_bf16x2(s.z, s.w));
  }
  __syncwarp();
  ptx::cluster_sync_relaxed();                     // nobody still reads this CTA's part
}

// `tiles` tiles; the contraction is split as far as the tiles' clusters still are on
// the GPU together and a CTA has four stages on average (they go out in equal runs,
// the last ranks' are shorter or empty): a second wave costs more than a larger split
// gains (60 tiles, 1536 channels, K 4096: 8.2 us by four CTAs a tile,
// 12.9 by five, whose 58 clusters leave two for later; 96 tiles 13.7 by three, 18.7
// by two).
template <int OP, bool I8, bool F32>
int launch_few(const CUtensorMap& ta, const CUtensorMap& tb, const RaggedArgs& p, int64_t tiles, int64_t nst,
               cudaStream_t s) {
  auto kern = ragged_few_kernel<OP, I8, F32>;
  static OncePerDevice once;
  static int residents[OncePerDevice::kDevices][9];  // by device and CTAs a cluster
  if (!once.run([&](int dev) {
        return cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)few_smem(I8)) == cudaSuccess &&
               resident_clusters(few_threads(I8), few_smem(I8), residents[dev]);
      }))
    return MGQ_ERR_CUDA;
  int dev = 0;
  cudaGetDevice(&dev);
  const int* resident = residents[dev];
  int split = 8;
  while (split > 1 && (tiles > resident[split] || nst / split < 4)) --split;
  if (tiles >= (1ll << 31)) return MGQ_ERR_INVALID_ARG;
  // int8: as many CTAs as are on the GPU at once take the tiles in turn, so that the
  // ring goes on over a tile's end (32 rows over 8 x [28672, 4096] 162 -> 151-154 us, 1000
  // rows over 256 x [512, 2048] 74 -> 64). bf16 tiles have twice the bytes, and the GPU's own order of
  // handing out CTAs serves them better (259 us against 263).
  const int64_t ctas = split > 1 ? tiles * split : I8 ? min(tiles, (int64_t)resident[1]) : tiles;
  return launch_after(kern, dim3((unsigned)ctas), few_threads(I8), few_smem(I8), split, s, ta, tb, p, split)
             ? MGQ_OK
             : MGQ_ERR_CUDA;
}

}  // namespace

int run_few(int op, bool i8, const CUtensorMap& ta, const CUtensorMap& tb, const RaggedArgs& p, cudaStream_t s) {
  const int64_t tiles = token_tiles(p.E, p.R, kFewTok) * ((p.M + 127) / 128);
  const int64_t nst = (p.C + (i8 ? kBK8 : 64) - 1) / (i8 ? kBK8 : 64);
  if (i8) return p.out_f32 ? launch_few<kFwd, true, true>(ta, tb, p, tiles, nst, s)
                           : launch_few<kFwd, true, false>(ta, tb, p, tiles, nst, s);
  if (op == kFwd) return p.out_f32 ? launch_few<kFwd, false, true>(ta, tb, p, tiles, nst, s)
                                   : launch_few<kFwd, false, false>(ta, tb, p, tiles, nst, s);
  return p.out_f32 ? launch_few<kDgrad, false, true>(ta, tb, p, tiles, nst, s)
                   : launch_few<kDgrad, false, false>(ta, tb, p, tiles, nst, s);
}

}  // namespace mgq
