// Host-side internals shared by the translation units of libmgq.
#pragma once
#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <atomic>
#include <mutex>

#include "mgq.h"

namespace mgq {

// Device address of the current device's error word (cached per device).
// Returns nullptr if it cannot be resolved.
int* error_word();

// Encodes a 2D row-major tiled tensor map of unsigned bytes: `inner` bytes per
// row (contiguous), `outer` rows with a pitch of `pitch` bytes; the box is
// box_inner x box_outer with 128-byte swizzling (box_inner == 128).
bool encode_tmap_u8_2d(CUtensorMap* map, const void* base, uint64_t inner, uint64_t outer, uint64_t pitch,
                       uint32_t box_inner, uint32_t box_outer);

// 2D row-major tensor map of 8-, 16- or 32-bit elements (elem_bytes 1, 2 or 4):
// `inner` elements per row, `outer` rows, pitch bytes; no swizzle, or with
// sw128 the 128-byte swizzle (box_inner * elem_bytes == 128).
bool encode_tmap_2d(CUtensorMap* map, const void* base, int elem_bytes, uint64_t inner, uint64_t outer,
                    uint64_t pitch, uint32_t box_inner, uint32_t box_outer, bool sw128 = false);

// 3D tensor map of 8-, 16- or 32-bit elements with the 128- or 64-byte swizzle
// (box[0] * elem_bytes is the one or the other): dims[0] elements contiguous, pitch1 bytes from
// one dims[1] index to the next, pitch2 bytes from one dims[2] index to the next.
// What a box covers outside the dims reads as zero and is not stored.
bool encode_tmap_swz_3d(CUtensorMap* map, const void* base, int elem_bytes, const uint64_t (&dims)[3],
                        uint64_t pitch1, uint64_t pitch2, const uint32_t (&box)[3]);

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

inline cudaStream_t as_stream(void* s) { return reinterpret_cast<cudaStream_t>(s); }

// The failure-detection options (mgq_set_gemm_option): whether producers issue
// no copies, and the limit of a pipeline wait (gemm.cu).
void debug_knobs(int* stall, uint64_t* wait_ns);

// Number of SMs of the current device (cached).
int num_sms();

// dst[c, r] = src[r, c] for r < *rows_used (or rows_cap when rows_used is
// null), c < cols; 64x64 byte tiles (routing.cu).
int launch_transpose_u8(const uint8_t* src, int64_t src_ld, uint8_t* dst, int64_t dst_ld, const int32_t* rows_used,
                        int64_t rows_cap, int64_t cols, cudaStream_t s);

// amax[g] = max |x| over each of G groups of per_group bf16 values (zeroes
// amax first; elementwise.cu).
int launch_amax_groups(const uint16_t* x, int64_t per_group, int64_t G, float* amax, cudaStream_t s);
// NVFP4 row-wise codes of x [rows, K] (rows_used on the device, or null) with
// s_g = 2688 / *amax, written to *s_out
int launch_quant_rows_nv(const uint16_t* x, int64_t rows, const int32_t* rows_used, int64_t K, uint8_t* codes,
                         uint8_t* scales, const float* amax, float* s_out, cudaStream_t s);

// Row-wise + column-wise quantisation in one pass (quant_tile.cu); q->col.data
// must be set. Per-tensor or MX scaling.
int rowcol_plain(const uint16_t* x, int64_t G, int64_t M, int64_t K, const mgq_qdesc* q, cudaStream_t s);
// row-wise and column-wise copies of a bf16 [rows_cap, C] matrix whose rows in
// use are *rows_used (one group: column copy [C, rows_cap]) (quant_tile.cu)
int rowcol_rows(const uint16_t* x, int64_t rows_cap, const int32_t* rows_used, int64_t C, const mgq_qdesc* q,
                cudaStream_t s);
int rowcol_swiglu(const uint16_t* gu, int64_t R_cap, int64_t F, const int32_t* rows_used, uint16_t* h_out,
                  const mgq_qdesc* q, cudaStream_t s);
int rowcol_dswiglu(const uint16_t* dh, const uint16_t* gu, int64_t R_cap, int64_t F, const int32_t* rows_used,
                   uint16_t* out, const mgq_qdesc* q, cudaStream_t s);

// Column-wise copies (MX or per-tensor) of the permuted X rows, with the
// row-wise codes too when `with_rows`, and column-wise copies only of
// dY = probs * dout rows, gathered through src_row (quant_tile.cu).
int gather_x_rowcol(const uint16_t* x, const int32_t* src_row, int k, int64_t H, int64_t R_cap,
                    const int32_t* rows_used, bool with_rows, const mgq_qdesc* q, cudaStream_t s);
int col_gather_dy(const uint16_t* dout, const float* probs, const int32_t* src_row, int k, int64_t H,
                  int64_t R_cap, const int32_t* rows_used, const mgq_qdesc* q, cudaStream_t s);

// NVFP4 weights with 16x16 blocks: row-wise [G*M, K/2] and (when col_codes
// is set) column-wise [G*K, M/2] codes with tiled ue4m3 scales; s_g per group
// from amax (written to s_out) (quant_tile.cu)
int quant_nv2d(const uint16_t* x, int64_t G, int64_t M, int64_t K, uint8_t* row_codes, uint8_t* row_scales,
               uint8_t* col_codes, uint8_t* col_scales, const float* amax, float* s_out, cudaStream_t s);

// n[c], c of 1 to 8: clusters of c CTAs of up to 256 threads and 128 registers that
// are on the GPU at once. They lie within a GPC, and what its SMs leave over differs
// (two CTAs an SM: 304, 152, 97, 74, 58, 46, 38 and 36). The runtime is asked about a
// kernel that does nothing: for one that allocates tensor memory it counts one CTA an SM.
bool resident_clusters(int threads, size_t smem, int* n);

// What a launcher sets and asks once per device (a static one for each kernel). run()
// calls prepare(dev) for the current device until it has returned true; one host thread
// at a time, and a caller that gets true sees all that prepare wrote.
class OncePerDevice {
 public:
  template <typename F>
  bool run(F prepare) {
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kDevices) return false;
    if (done_[dev].load(std::memory_order_acquire)) return true;
    std::lock_guard<std::mutex> lk(mu_);
    if (done_[dev].load(std::memory_order_relaxed)) return true;
    if (!prepare(dev)) {
      (void)cudaGetLastError();
      return false;
    }
    done_[dev].store(true, std::memory_order_release);
    return true;
  }
  static constexpr int kDevices = 64;

 private:
  std::mutex mu_;
  std::atomic<bool> done_[kDevices]{};
};

// A launch that may start while the kernel before it in the stream still runs
// (programmatic dependent launch): such a kernel reads what others wrote, and
// writes, only after griddepcontrol.wait. `cluster`: CTAs along x, 1 for none.
template <typename... P, typename... A>
bool launch_after(void (*kern)(P...), dim3 grid, int threads, size_t smem, int cluster, cudaStream_t s, A... args) {
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  at[1].id = cudaLaunchAttributeClusterDimension;
  at[1].val.clusterDim.x = cluster;
  at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cfg.attrs = at;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  if (cudaLaunchKernelEx(&cfg, kern, args...) == cudaSuccess) return true;
  (void)cudaGetLastError();
  return false;
}

}  // namespace mgq

#define MGQ_CHECK_ARG(cond)                 \
  do {                                      \
    if (!(cond)) return MGQ_ERR_INVALID_ARG; \
  } while (0)

#define MGQ_LAUNCH_CHECK()                           \
  do {                                               \
    if (cudaPeekAtLastError() != cudaSuccess) {      \
      (void)cudaGetLastError();                      \
      return MGQ_ERR_CUDA;                           \
    }                                                \
  } while (0)
