// bf16 products grouped by expert over ragged groups: group e is the rows
// [offsets[e], offsets[e+1]), any row numbers, no padding.
//
//   fwd    Y[r, n]    = sum_k X[r, k] W[e, n, k]
//   dgrad  dX[r, k]   = sum_n dY[r, n] W[e, n, k]
//   wgrad  dW[e, n, k] = beta dW[e, n, k] + sum_{r in e} dY[r, n] X[r, k]
//
// (The unquantised product that the routed-expert recipes are compared with:
// `grouped_mm` in "float8 moe training conversion API prototype", pytorch/ao
// PR #2275, and the BF16 runs of Megatron-LM issue #1152.)
//
// Design. Two SMs share a tile (cta_group::2): M = 256 on the weights' side,
// 128 rows an SM, and up to 256 tokens on the N side, whose extent an MMA takes
// in steps of 32 from its instruction descriptor: the last tile of a group
// costs by the rows it has, and a group's first row is any row, because the row
// coordinate of a TMA box has no alignment. The accumulator then holds channels
// as lanes and tokens as columns; the epilogue stores only the group's own rows:
// runs of 32 tokens through shared memory and the TMA, shorter ones from registers
// (bf16: 8 x 8 blocks transposed between lanes, 16 bytes of a token at a time).
// The transposed weights of dgrad and both operands of wgrad are read MN-major
// by the tensor cores. wgrad contracts over the tokens: rows of the last 16-row
// step that belong to the next group are zeroed in shared memory, in both
// operands (0 times a NaN of another group is a NaN).
//
// Bound by the tensor cores (active 97% of the time at 8192 rows of 4 x [8192, 4096])
// and, for long calls, by the power cap. Measured: 8192^3 forward 572-587 us (1870-1920
// TFLOP/s), dgrad 574-603, wgrad 588-610 on a card that was idle before, 6 to 9% more on
// one that was not; 8024 rows over 128 x [1536, 2048] dgrad 131 us (6.6 TB/s), wgrad into
// 128 x [2048, 768] float32 133-136 us (6.3 TB/s, the writes). With beta that call takes
// 637 us: the old result comes by loads of 16 bytes a lane, each in its own row, after
// the sums are complete. wgrad gives a tile all of its group's rows, so few tiles leave
// most of the GPU idle (one expert of [1024, 1024], 32768 rows: 16 tiles, 149 us).
#include "ragged.cuh"

namespace mgq {
namespace {

constexpr int kBK = 64;                            // elements of the contraction a stage (128 bytes)
constexpr uint32_t kOpBytes = 128 * 128;           // one operand's share of an SM a stage
constexpr uint32_t kOutSlot = 32 * 128;            // wgrad: a warp's store staging
__host__ __device__ constexpr uint32_t slot_of(int op) { return op == kWgrad ? kOutSlot : kTokSlot; }
// float32 results: the tensor cores cut each sum off rather than round it, and
// the error grows with every K=16 step (1.5e-8 a step, relative: 4.4e-6 after a
// contraction of 4096, which a float32 result shows and a bf16 one does not).
// So after kPromote stages the partial sum moves to registers of the epilogue,
// where it is added with rounding, while the other accumulator goes on. (168 registers
// a thread, and a few spilled: 20 bytes stored and 52 loaded, wgrad 44 and 196. 8192^3
// 587 -> 700 us, wgrad 610 -> 672.)
constexpr int kPromote = 8;
__host__ __device__ constexpr int stages_of(int op) { return op == kWgrad ? 5 : 6; }
__host__ __device__ constexpr int threads_of(int op) { return op == kWgrad ? 352 : 320; }
__host__ __device__ constexpr size_t smem_of(int op) {
  return 1024 + stages_of(op) * 2 * (size_t)kOpBytes + 8 * slot_of(op) + 256 + 2 * (kMaxE + 8) * 4;
}
static_assert(smem_of(kFwd) <= 232448 && smem_of(kWgrad) <= 232448, "shared memory");

template <int OP, bool F32>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(threads_of(OP), 1)
    ragged_pair_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                       const __grid_constant__ CUtensorMap tmS, const __grid_constant__ CUtensorMap tmO,
                       const RaggedArgs p) {
  constexpr int ST = stages_of(OP);
  constexpr bool kAmn = OP != kFwd, kBmn = OP == kWgrad;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = ptx::smem_u32(smem_raw);
  uint8_t* sA = smem_raw + (((raw + 1023u) & ~1023u) - raw);
  uint8_t* sB = sA + ST * kOpBytes;
  uint8_t* sOut = sB + ST * kOpBytes;
  uint64_t* full = reinterpret_cast<uint64_t*>(sOut + 8 * slot_of(OP));
  uint64_t* empty = full + ST;
  uint64_t* tmem_full = empty + ST;      // [2]
  uint64_t* tmem_empty = tmem_full + 2;  // [2]
  uint64_t* mask_go = tmem_empty + 2;    // wgrad: the last stage has landed in both SMs
  uint64_t* mask_done = mask_go + 1;     // its foreign rows are zero
  uint64_t* drained = mask_done + 1;     // after a wait ran out: the MMAs issued have finished
  uint32_t* s_tmem = reinterpret_cast<uint32_t*>(drained + 1);
  volatile int* s_abort = reinterpret_cast<volatile int*>(s_tmem + 1);
  int* s_bad = reinterpret_cast<int*>(s_tmem + 2);
  int32_t* s_off = reinterpret_cast<int32_t*>(full + 32);
  int32_t* s_cum = s_off + (kMaxE + 8);

  const int warp = __shfl_sync(0xFFFFFFFFu, (int)(threadIdx.x >> 5), 0);   // (known to be uniform)
  const uint32_t lane = threadIdx.x & 31;
  const uint32_t rank = ptx::cluster_ctarank();
  const bool leader = rank == 0;
  const int64_t pair = blockIdx.x >> 1, npairs = gridDim.x >> 1;

  if (threadIdx.x == 0) {
    for (int s = 0; s < ST; ++s) {
      ptx::mbar_init(&full[s], 1);
      ptx::mbar_init(&empty[s], 1);
    }
    for (int a = 0; a < 2; ++a) {
      ptx::mbar_init(&tmem_full[a], 1);
      ptx::mbar_init(&tmem_empty[a], 2 * 8);      // one arrival per epilogue warp of each CTA
    }
    ptx::mbar_init(mask_go, 1);
    ptx::mbar_init(mask_done, 2);
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
    const bool ok = load_groups(p, s_off, s_cum, lane);
    if (lane == 0) {
      *s_bad = ok ? 0 : 1;
      if (!ok) report(p.err, MGQ_ERR_INVALID_ARG);
    }
  }
  __syncthreads();
  ptx::tc_fence_before();
  ptx::cluster_sync();                 // both CTAs' barriers initialised, tensor memory allocated
  ptx::tc_fence_after();
  const uint32_t tmem = *s_tmem;
  const bool run = *s_bad == 0;

  if (run && warp == 0 && !p.stall && ptx::elect_one()) {
    // ------------------------------------------------------------ producer (both CTAs)
    int ecur = 0;
    uint32_t it = 0, st = 0, ph = 0;
    RaggedTile tl;
    for (int64_t t = pair; !*s_abort && ragged_tile<OP>(s_off, s_cum, p, t, ecur, tl); t += npairs) {
      // this CTA's half of the tokens: one box of 128 rows, or boxes of 32
      const int half = OP == kWgrad ? 128 : (tl.n + 31) / 32 * 16;
      const int boxes = half == 128 ? 0 : (half + (int)kSmallBox - 1) / (int)kSmallBox;
      const uint32_t bytes = 2 * (kOpBytes + (boxes ? boxes * kSmallBox * 128 : kOpBytes));
      for (int s = 0; s < tl.nst; ++s, ++it) {
        if (*s_abort) break;
        if (!ptx::mbar_wait(&empty[st], ph ^ 1, p.wait_ns)) {
          report(p.err, MGQ_ERR_TIMEOUT);
          *s_abort = 1;
          break;
        }
        if (leader) ptx::mbar_arrive_expect_tx(&full[st], bytes);
        const uint32_t bar0 = ptx::mapa_shared(ptx::smem_u32(&full[st]), 0);
        uint8_t* a = sA + st * kOpBytes;
        uint8_t* b = sB + st * kOpBytes;
        const int32_t kx = s * kBK;
        const int32_t am = (int32_t)(tl.m0 + 128 * rank);
        if (OP == kFwd) {
          ptx::tma_load_3d_pair(a, &tmA, bar0, kx, am, tl.e);
        } else {                                     // two chunks of 64 along M
          const int32_t y = OP == kDgrad ? kx : tl.row0 + kx, z = OP == kDgrad ? tl.e : 0;
          ptx::tma_load_3d_pair(a, &tmA, bar0, am, y, z);
          ptx::tma_load_3d_pair(a + kOpBytes / 2, &tmA, bar0, am + 64, y, z);
        }
        if (OP == kWgrad) {
          const int32_t x = (int32_t)(tl.c0 + 128 * rank);
          ptx::tma_load_3d_pair(b, &tmB, bar0, x, tl.row0 + kx, 0);
          ptx::tma_load_3d_pair(b + kOpBytes / 2, &tmB, bar0, x + 64, tl.row0 + kx, 0);
        } else {
          const int32_t r = tl.row0 + half * (int)rank;
          if (!boxes) ptx::tma_load_3d_pair(b, &tmB, bar0, kx, r, 0);
          for (int i = 0; i < boxes; ++i)
            ptx::tma_load_3d_pair(b + i * kSmallBox * 128, &tmS, bar0, kx, r + i * (int)kSmallBox, 0);
        }
        if (++st == ST) st = 0, ph ^= 1;
      }
    }
    // after a wait that ran out: no copy may still be on its way when the CTA
    // leaves. (The leader's barriers count both CTAs' copies.)
    if (*s_abort && leader)
      for (uint32_t i = it > ST ? it - ST : 0; i < it; ++i) ptx::mbar_wait(&full[i % ST], (i / ST) & 1, p.wait_ns);
  } else if (run && leader && warp == 1 && ptx::elect_one()) {
    // ------------------------------------------------------------ MMA issuer (CTA 0)
    int ecur = 0;
    uint32_t st = 0, ph = 0, tc = 0, masks = 0;
    RaggedTile tl;
    const uint32_t sA0 = ptx::smem_u32(sA), sB0 = ptx::smem_u32(sB);
    bool ok = true;
    for (int64_t t = pair; ok && ragged_tile<OP>(s_off, s_cum, p, t, ecur, tl); t += npairs) {
      if (tl.nst == 0) continue;
      const uint32_t N = OP == kWgrad ? 256u : (uint32_t)(tl.n + 31) / 32 * 32;
      const uint32_t idesc = ptx::idesc_f16(1, 256, N) | ptx::idesc_mn_major(kAmn, kBmn);
      uint32_t a = 0;
      for (int s = 0; s < tl.nst; ++s) {
        const bool first = s == 0 || (F32 && s % kPromote == 0);   // of an accumulator
        if (first) {
          a = tc & 1;
          ok = !*s_abort && ptx::mbar_wait(&tmem_empty[a], ((tc >> 1) & 1) ^ 1, p.wait_ns);
          if (!ok) break;
        }
        ok = !*s_abort && ptx::mbar_wait(&full[st], ph, p.wait_ns);
        int steps = kBK / 16;
        if (OP == kWgrad && s == tl.nst - 1 && ok) {
          const int rows = tl.n - s * kBK;
          steps = (rows + 15) / 16;
          if (rows % 16) {
            ptx::mbar_arrive_pair(ptx::mapa_shared(ptx::smem_u32(mask_go), 0));
            ptx::mbar_arrive_pair(ptx::mapa_shared(ptx::smem_u32(mask_go), 1));
            ok = ptx::mbar_wait(mask_done, masks++ & 1, p.wait_ns);
          }
        }
        if (!ok) break;
        ptx::tc_fence_after();
        const uint64_t ad = kAmn ? ptx::sdesc_mnmajor_sw128_chunks(sA0 + st * kOpBytes, kOpBytes / 2)
                                 : ptx::sdesc_kmajor_sw128(sA0 + st * kOpBytes);
        const uint64_t bd = kBmn ? ptx::sdesc_mnmajor_sw128_chunks(sB0 + st * kOpBytes, kOpBytes / 2)
                                 : ptx::sdesc_kmajor_sw128(sB0 + st * kOpBytes);
        // a K=16 step: 32 bytes along a K-major row, 16 rows (2048 bytes) of an MN-major tile
        constexpr uint64_t da = kAmn ? 128 : 2, db = kBmn ? 128 : 2;
        for (int kk = 0; kk < steps; ++kk)
          ptx::mma_f16_pair(tmem + a * kTile, ad + kk * da, bd + kk * db, idesc, (!first || kk > 0) ? 1u : 0u);
        ptx::mma_commit_pair(&empty[st], 0x3);        // frees the stage in both CTAs
        if (++st == ST) st = 0, ph ^= 1;
        if (s == tl.nst - 1 || (F32 && s % kPromote == kPromote - 1)) {
          ptx::mma_commit_pair(&tmem_full[a], 0x3);
          ++tc;
        }
      }
    }
    if (!ok) {
      report(p.err, MGQ_ERR_TIMEOUT);
      *s_abort = 1;
      ptx::mma_commit_pair(drained, 0x1);             // the MMAs issued so far finish before the CTA leaves
      ptx::mbar_wait(drained, 0, p.wait_ns);
    }
  } else if (run && warp >= 2 && warp < 10) {
    // ------------------------------------------------------------ epilogue (both CTAs)
    const uint32_t q = warp & 3;
    const uint32_t half = (uint32_t)(warp - 2) >> 2;
    const uint32_t empty0 = ptx::mapa_shared(ptx::smem_u32(&tmem_empty[0]), 0);
    const uint32_t empty1 = ptx::mapa_shared(ptx::smem_u32(&tmem_empty[1]), 0);
    uint8_t* slot = sOut + (warp - 2) * slot_of(OP);
    int ecur = 0;
    uint32_t tc = 0;
    RaggedTile tl;
    bool ok = true;
    for (int64_t t = pair; ok && ragged_tile<OP>(s_off, s_cum, p, t, ecur, tl); t += npairs) {
      const int64_t m0 = tl.m0 + 128 * rank + 32 * q;       // this warp's 32 rows of the M side
      // its columns: four runs of 32 (the rows' products: every second run, so that
      // a short tile's tokens are shared by both warps)
      const int width = OP == kWgrad ? (int)min((int64_t)kTile, p.C - tl.c0) : tl.n;
      auto col = [&](int i) { return OP == kWgrad ? 128 * (int)half + 32 * i : 32 * (int)half + 64 * i; };
      float v[F32 ? 4 : 1][32];
      const int parts = tl.nst == 0 ? 0 : F32 ? (tl.nst + kPromote - 1) / kPromote : 1;
      if (F32 && parts == 0) {
#pragma unroll
        for (int i = 0; i < (F32 ? 4 : 1); ++i)
#pragma unroll
          for (int j = 0; j < 32; ++j) v[i][j] = 0.0f;
      }
      // the next accumulator, and its release once it is read
      auto wait_acc = [&]() {
        bool got = *s_abort == 0;
        got = got && ptx::mbar_wait(&tmem_full[tc & 1], (tc >> 1) & 1, p.wait_ns);
        if (!__all_sync(0xFFFFFFFFu, got)) {
          report(p.err, MGQ_ERR_TIMEOUT);
          *s_abort = 1;
          return false;
        }
        ptx::tc_fence_after();
        return true;
      };
      auto release_acc = [&]() {
        ptx::tc_fence_before();
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive_pair(tc & 1 ? empty1 : empty0);
        ++tc;
      };
      auto load = [&](int i, float (&d)[32], bool add) {
#pragma unroll
        for (int h = 0; h < 32; h += 16) {
          uint32_t r[16];
          ptx::tmem_ld_32x32b_x16(tmem + (tc & 1) * kTile + ((q * 32) << 16) + col(i) + h, r);
          ptx::tmem_ld_wait();
#pragma unroll
          for (int j = 0; j < 16; ++j) d[h + j] = add ? d[h + j] + __uint_as_float(r[j]) : __uint_as_float(r[j]);
        }
      };
      if (F32) {
        for (int part = 0; part < parts; ++part) {
          if (!(ok = wait_acc())) break;
#pragma unroll
          for (int i = 0; i < (F32 ? 4 : 1); ++i)
            if (col(i) < width) load(i, v[i], part > 0);
          release_acc();
        }
        if (!ok) break;
      } else if (parts) {
        if (!(ok = wait_acc())) break;
      }
      if (OP != kWgrad) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          if (col(i) >= width) break;
          float(&x)[32] = v[F32 ? i : 0];
          if (!F32) load(i, x, false);
          if (width - col(i) >= 32 && m0 < p.M) send_tokens<F32>(&tmO, slot, x, tl.row0 + col(i), (int32_t)m0, lane);
          else store_tokens<F32>(p.out, p.ldo, x, (int64_t)tl.row0 + col(i), width - col(i), m0, p.M, lane);
        }
      } else if (m0 < p.M) {
        // staged rows of 128 bytes: 32 float32 columns, or 64 of bf16
#pragma unroll
        for (int i = 0; i < 4; i += F32 ? 1 : 2) {
          const int c = col(i);
          if (c >= width) break;
          uint32_t w[32];
          if (F32) {
            if (p.beta != 0.0f && m0 + lane < p.M) {
              const float* old = static_cast<const float*>(p.out) + ((int64_t)tl.e * p.M + m0 + lane) * p.C + tl.c0 + c;
#pragma unroll
              for (int j = 0; j < 32; j += 4) {
                if (c + j >= width) break;                  // (the width is a multiple of 8)
                const float4 o = *reinterpret_cast<const float4*>(old + j);
                float* x = v[F32 ? i : 0] + j;
                x[0] = fmaf(p.beta, o.x, x[0]);
                x[1] = fmaf(p.beta, o.y, x[1]);
                x[2] = fmaf(p.beta, o.z, x[2]);
                x[3] = fmaf(p.beta, o.w, x[3]);
              }
            }
#pragma unroll
            for (int j = 0; j < 32; ++j) w[j] = __float_as_uint(v[F32 ? i : 0][j]);
          } else {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
#pragma unroll
              for (int j = 0; j < 32; ++j) v[0][j] = 0.0f;
              if (parts) load(i + h, v[0], false);
#pragma unroll
              for (int j = 0; j < 16; ++j) w[16 * h + j] = pack_bf16x2(v[0][2 * j], v[0][2 * j + 1]);
            }
          }
          if (lane == 0) ptx::bulk_wait_read0();            // the store before has read the staging slot
          __syncwarp();
#pragma unroll
          for (int j = 0; j < 8; ++j)
            *reinterpret_cast<uint4*>(slot + lane * 128 + ((j ^ (lane & 7)) << 4)) =
                make_uint4(w[4 * j], w[4 * j + 1], w[4 * j + 2], w[4 * j + 3]);
          ptx::fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) {
            ptx::tma_store_3d(&tmO, slot, (int32_t)(tl.c0 + c), (int32_t)m0, tl.e);
            ptx::bulk_commit();
          }
        }
      }
      if (!F32 && parts) release_acc();
    }
    if (lane == 0) ptx::bulk_wait0();                       // this warp's stores are complete
  } else if (OP == kWgrad && run && warp == 10) {
    // ------------------------------------------------------------ foreign rows of a group's last step
    int ecur = 0;
    uint32_t it = 0, masks = 0;
    RaggedTile tl;
    const uint32_t done0 = ptx::mapa_shared(ptx::smem_u32(mask_done), 0);
    for (int64_t t = pair; ragged_tile<OP>(s_off, s_cum, p, t, ecur, tl); t += npairs) {
      it += tl.nst;
      const int rows = tl.n - (tl.nst - 1) * kBK;
      if (tl.nst == 0 || rows % 16 == 0) continue;
      // (a tile before this one can take long: this wait is for a stage, so it
      // is repeated until the pipeline itself has given up)
      bool got = false;
      while (!got && !*s_abort) got = ptx::mbar_wait(mask_go, masks & 1, 1000000);
      if (!__all_sync(0xFFFFFFFFu, got)) break;
      ++masks;
      const uint32_t st = (it - 1) % ST;
      for (int r = rows; r < (rows + 15) / 16 * 16; ++r) {
        // a row is 128 bytes in each of the operands' two chunks
        uint8_t* base = (lane < 16 ? sA : sB) + st * kOpBytes + (lane & 8 ? kOpBytes / 2 : 0);
        *reinterpret_cast<uint4*>(base + r * 128 + (lane & 7) * 16) = make_uint4(0, 0, 0, 0);
      }
      ptx::fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive_pair(done0);
    }
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

template <int OP, bool F32>
int launch_pair(const CUtensorMap& ta, const CUtensorMap& tb, const CUtensorMap& ts, const CUtensorMap& to,
                const RaggedArgs& p, int64_t max_tiles, cudaStream_t s) {
  auto kern = ragged_pair_kernel<OP, F32>;
  static OncePerDevice once;
  if (!once.run([&](int) {
        return cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem_of(OP)) == cudaSuccess;
      }))
    return MGQ_ERR_CUDA;
  const int64_t pairs = min((int64_t)(num_sms() / 2), max_tiles);
  return launch_after(kern, dim3((unsigned)(2 * max(pairs, (int64_t)1))), threads_of(OP), smem_of(OP), 1, s, ta, tb, ts, to, p)
             ? MGQ_OK
             : MGQ_ERR_CUDA;
}

// What every entry point checks: sizes, pitches, alignment.
int check_ragged(const void* a, int64_t lda, int64_t wa, const void* b, int64_t ldb, int64_t wb, const int32_t* offsets,
                 int E, int64_t R, int64_t N, int64_t K, const void* out, int out_dtype) {
  MGQ_CHECK_ARG(E >= 1 && E <= kMaxE && R >= 0 && R < (1ll << 31) - 512 && N > 0 && K > 0);
  MGQ_CHECK_ARG(N % 8 == 0 && K % 8 == 0 && N < (1ll << 31) - 512 && K < (1ll << 31) - 512);
  MGQ_CHECK_ARG(offsets || E == 1);
  MGQ_CHECK_ARG(out_dtype == MGQ_OUT_BF16 || out_dtype == MGQ_OUT_F32);
  MGQ_CHECK_ARG((reinterpret_cast<uintptr_t>(offsets) & 3u) == 0 && aligned16(out));
  MGQ_CHECK_ARG(lda >= wa && lda % 8 == 0 && ldb >= wb && ldb % 8 == 0 && lda < (1ll << 38) && ldb < (1ll << 38));
  MGQ_CHECK_ARG(aligned16(a) && aligned16(b) && (R == 0 || (a && b && out)));
  return MGQ_OK;
}

void fill_knobs(RaggedArgs* p) { debug_knobs(&p->stall, &p->wait_ns); }

// fwd and dgrad: rows of `in` [R, C] by the weights, result columns M.
template <int OP>
int run_rows(const void* in, int64_t ldi, const void* w, const int32_t* offsets, int E, int64_t R, int64_t N, int64_t K,
             void* out, int64_t ldo, int out_dtype, void* stream) {
  const int64_t M = OP == kFwd ? N : K, C = OP == kFwd ? K : N;
  int rc = check_ragged(in, ldi, C, w, K, K, offsets, E, R, N, K, out, out_dtype);
  if (rc != MGQ_OK) return rc;
  MGQ_CHECK_ARG(ldo >= M && ldo % 8 == 0 && ldo < (1ll << 38));
  if (R == 0) return MGQ_OK;
  RaggedArgs p{};
  p.err = error_word();
  if (!p.err) return MGQ_ERR_CUDA;
  p.offsets = offsets;
  p.E = E;
  p.R = R;
  p.M = M;
  p.C = C;
  p.out = out;
  p.ldo = ldo;
  p.out_f32 = out_dtype == MGQ_OUT_F32;
  fill_knobs(&p);
  CUtensorMap ta, tb, ts, to;
  const uint64_t u = 2;
  p.bk = kBK;
  if (few_rows(E, R, M, false)) {
    if (!encode_tmap_swz_3d(&ta, w, 2, {(uint64_t)K, (uint64_t)N, (uint64_t)E}, K * u, N * K * u,
                              {64, OP == kFwd ? 128u : 64u, 1}) ||
        !encode_tmap_swz_3d(&ts, in, 2, {(uint64_t)C, (uint64_t)R, 1}, ldi * u, R * ldi * u, {64, kFewBox, 1}))
      return MGQ_ERR_CUDA;
    return run_few(OP, false, ta, ts, p, as_stream(stream));
  }
  if (!encode_tmap_swz_3d(&ta, w, 2, {(uint64_t)K, (uint64_t)N, (uint64_t)E}, K * u, N * K * u,
                            {64, OP == kFwd ? 128u : 64u, 1}) ||
      !encode_tmap_swz_3d(&tb, in, 2, {(uint64_t)C, (uint64_t)R, 1}, ldi * u, R * ldi * u, {64, 128, 1}) ||
      !encode_tmap_swz_3d(&ts, in, 2, {(uint64_t)C, (uint64_t)R, 1}, ldi * u, R * ldi * u, {64, kSmallBox, 1}) ||
      !encode_out(&to, out, R, M, ldo, p.out_f32))
    return MGQ_ERR_CUDA;
  const int64_t tiles = token_tiles(E, R, kTile) * ((M + kTile - 1) / kTile);
  p.bk = kBK;
  return p.out_f32 ? launch_pair<OP, true>(ta, tb, ts, to, p, tiles, as_stream(stream))
                   : launch_pair<OP, false>(ta, tb, ts, to, p, tiles, as_stream(stream));
}

}  // namespace
}  // namespace mgq

using namespace mgq;

extern "C" {

int mgq_ragged_gemm_fwd(const void* x_bf16, int64_t ldx, const void* w_bf16, const int32_t* offsets, int E, int64_t R,
                        int64_t N, int64_t K, void* y, int64_t ldy, int out_dtype, void* stream) {
  return run_rows<kFwd>(x_bf16, ldx, w_bf16, offsets, E, R, N, K, y, ldy, out_dtype, stream);
}

int mgq_ragged_gemm_dgrad(const void* dy_bf16, int64_t lddy, const void* w_bf16, const int32_t* offsets, int E,
                          int64_t R, int64_t N, int64_t K, void* dx, int64_t lddx, int out_dtype, void* stream) {
  return run_rows<kDgrad>(dy_bf16, lddy, w_bf16, offsets, E, R, N, K, dx, lddx, out_dtype, stream);
}

int mgq_ragged_gemm_wgrad(const void* dy_bf16, int64_t lddy, const void* x_bf16, int64_t ldx, const int32_t* offsets,
                          int E, int64_t R, int64_t N, int64_t K, float beta, void* dw, int out_dtype, void* stream) {
  int rc = check_ragged(dy_bf16, lddy, N, x_bf16, ldx, K, offsets, E, R, N, K, dw, out_dtype);
  if (rc != MGQ_OK) return rc;
  MGQ_CHECK_ARG(beta == 0.0f || out_dtype == MGQ_OUT_F32);
  MGQ_CHECK_ARG(beta == beta && dw);
  const int64_t u = out_dtype == MGQ_OUT_F32 ? 4 : 2;
  if (R == 0 && beta == 1.0f) return MGQ_OK;
  RaggedArgs p{};
  p.err = error_word();
  if (!p.err) return MGQ_ERR_CUDA;
  p.offsets = offsets;
  p.E = E;
  p.R = R;
  p.M = N;
  p.C = K;
  p.out = dw;
  p.out_f32 = out_dtype == MGQ_OUT_F32;
  p.beta = beta;
  fill_knobs(&p);
  CUtensorMap ta, tb, to;
  // (no rows: maps that no load uses, the groups' results are beta times what they were)
  const uint64_t rows = R > 0 ? R : 1;
  if (!encode_tmap_swz_3d(&ta, R > 0 ? dy_bf16 : dw, 2, {(uint64_t)N, rows, 1}, lddy * 2, rows * lddy * 2,
                            {64, 64, 1}) ||
      !encode_tmap_swz_3d(&tb, R > 0 ? x_bf16 : dw, 2, {(uint64_t)K, rows, 1}, ldx * 2, rows * ldx * 2,
                            {64, 64, 1}) ||
      !encode_tmap_swz_3d(&to, dw, (int)u, {(uint64_t)K, (uint64_t)N, (uint64_t)E}, K * u, N * K * u,
                            {(uint32_t)(128 / u), 32, 1}))
    return MGQ_ERR_CUDA;
  const int64_t tiles = (int64_t)E * ((N + kTile - 1) / kTile) * ((K + kTile - 1) / kTile);
  p.bk = kBK;
  return p.out_f32 ? launch_pair<kWgrad, true>(ta, tb, tb, to, p, tiles, as_stream(stream))
                   : launch_pair<kWgrad, false>(ta, tb, tb, to, p, tiles, as_stream(stream));
}

}  // extern "C"
