// qk_internal.h -- host-side declarations shared by the library's translation
// units (launchers, status words).  Not part of the public C ABI.
#pragma once

#include <atomic>
#include <cstdint>
#include <cuda_runtime.h>

#include "../../include/qk.h"

namespace qk {

enum QType : int { kQ4K = 0, kQ6K = 1 };

constexpr int kQK = 256;
constexpr int kQ4KBytes = 144;
constexpr int kQ6KBytes = 210;

inline int64_t block_bytes(QType t) { return t == kQ4K ? kQ4KBytes : kQ6KBytes; }

// Host state that CUDA keeps per device (function attributes, SM counts,
// occupancy answers) is cached per device index, for processes that drive
// several GPUs.
constexpr int kMaxDevices = 64;

// The calling thread's current device, or -1 if it cannot be read or is out
// of range.
int current_device();

// The current device's SM count (queried once per device).
int device_sms();

// One bit per device: set once that device's one-time setup has succeeded.
class PerDeviceFlag {
 public:
  bool done(int dev) const { return dev >= 0 && ((bits_.load(std::memory_order_acquire) >> dev) & 1u); }
  void mark(int dev) {
    if (dev >= 0) bits_.fetch_or(uint64_t(1) << dev, std::memory_order_release);
  }

 private:
  std::atomic<uint64_t> bits_{0};
};

// Launch a kernel whose CTAs may be scheduled while the kernel before it on the
// stream finishes (they call dependent_wait before touching memory), in
// clusters of `cluster` CTAs along x.
template <typename... Params, typename... Args>
cudaError_t launch_dependent(void (*kernel)(Params...), dim3 grid, unsigned threads, size_t smem, unsigned cluster,
                             cudaStream_t s, const Args&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  at[1].id = cudaLaunchAttributeClusterDimension;
  at[1].val.clusterDim.x = cluster;
  at[1].val.clusterDim.y = 1;
  at[1].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

// Each translation unit with kernels that can time out owns one device status
// word; these read it (after the stream has been synchronised) and clear it.
// Status bit of a copy that a debug build (QK_DEBUG) skipped (qk_device.cuh).
#ifndef QK_DEV_BAD_COPY
#define QK_DEV_BAD_COPY 4u
#endif
uint32_t dequant_take_status();
uint32_t gemv_take_status();
uint32_t gemm_take_status();

// Launchers.  Arguments are already validated; they return cudaGetLastError().
cudaError_t launch_dequant(QType t, const void* blocks, int64_t n_blocks, float* out, cudaStream_t s);
cudaError_t launch_gemv(QType t, const void* W, const uint16_t* x, float* y, int64_t N, int64_t K,
                        cudaStream_t s);
cudaError_t launch_gemm(QType t, const void* W, const void* W_up, const uint16_t* x, void* y, int64_t M,
                        int64_t N, int64_t K, bool gateup, cudaStream_t s);

// The tensor-core GEMM's launch plan for an M x N problem (host only; the
// fields mirror qk_gemm_plan_info).  False if no plan exists.
struct GemmPlanInfo {
  int token_tile, x_stages, a_stages, packed_stages, a_in_tmem, tmem_cols, smem_bytes, max_ctas_per_sm;
};
bool gemm_plan(QType t, bool gateup, int64_t M, int64_t N, GemmPlanInfo* info);

// RMSNorm rows into an fp16 buffer (problems the GEMV does not take):
// out[m][k] = fp16(x[m][k] / sqrt(mean_k x[m][k]^2 + eps) * gamma[k]).
cudaError_t launch_rmsnorm_rows(const uint16_t* x, const uint16_t* gamma, float eps, uint16_t* out, int64_t M,
                                int64_t K, cudaStream_t s);

// Residual addition + RMSNorm (qk_add_rmsnorm: xhat set; qk_add_rmsnorm_q8: xq
// and xd set); arguments validated.
cudaError_t launch_add_rmsnorm(const void* residual, bool f32, const float* delta, const uint16_t* gamma, float eps,
                               void* residual_out, uint16_t* xhat, int8_t* xq, float* xd, int64_t M, int64_t K,
                               cudaStream_t s);

// Rotary positions and the KV-cache rows (qk_rope_kv_append); arguments validated.
struct RopeArgs {
  const float *q, *k, *v;
  const double* inv_freq;
  uint16_t *q_out, *k_cache, *v_cache;
  int64_t M, pos0, Lmax;
  int H, Hkv, D, n_rot, half;
  float magnitude;
};
cudaError_t launch_rope_kv(const RopeArgs& a, cudaStream_t s);

// The same with an RMSNorm of each head in front (qk_norm_rope_kv_append; gammas
// may be null) and, where k_q4 is set, the rows in 4 bits instead
// (qk_norm_rope_kv_append_q4): 8 values a word of k_q4 / v_q4, (d, m) as two fp16
// a word of k_dm / v_dm.  Arguments validated.
struct NormRopeArgs {
  RopeArgs rope;
  const uint16_t *q_gamma, *k_gamma;
  float eps;
  uint32_t *k_q4, *v_q4, *k_dm, *v_dm;
};
cudaError_t launch_norm_rope(const NormRopeArgs& a, cudaStream_t s);

// Log probabilities, entropy and top alternatives (qk_logprobs); arguments validated.
struct LogprobArgs {
  const float* logits;
  const int32_t* tokens;
  float *logprob, *entropy, *top_logprobs;
  int32_t* top_ids;
  int64_t M;
  int V, top_n;
};
cudaError_t launch_logprobs(const LogprobArgs& a, cudaStream_t s);

// A token from each row of logits (qk_sample); arguments validated.
struct SampleArgs {
  const float *logits, *u;
  int32_t* token;
  float* logprob;
  int32_t* kept;
  int64_t M;
  int V, top_k;
  float temperature, top_p, min_p;
};
cudaError_t launch_sample(const SampleArgs& a, cudaStream_t s);

// The built-in scratch of qk_rmsnorm_matmul_batch_static (bytes) and its
// device address on the current device (looked up once per device).
constexpr size_t kStaticScratchBytes = size_t(8) << 20;
cudaError_t static_scratch_address(void** out);

// Encode a tiled TMA tensor map of fp16 elements into `out` (a CUtensorMap,
// 64 bytes): `rank` dimensions innermost first, the byte strides of
// dimensions 1.. (rank - 1 of them), the box, and a 128-byte swizzle or none.
// Elements outside the dimensions read as zero.  False if the driver refuses.
bool encode_tensor_map_f16(void* out, const void* base, int rank, const uint64_t* dims, const uint64_t* strides,
                           const uint32_t* box, bool swizzle128);

// GQA attention (qk_gqa_attention); arguments validated.  Device status word.
cudaError_t launch_gqa_attention(const uint16_t* q, const uint16_t* kc, const uint16_t* vc, float* out, int64_t M,
                                 int H, int Hkv, int64_t pos0, int64_t Lmax, float scale, cudaStream_t s);
// The same with a window and sinks, fp16 out (qk_gqa_attention_window), and its
// decode step (window and sinks at most pos0 + 1, not both 0).
cudaError_t launch_attn_window_decode(const uint16_t* q, const uint16_t* kc, const uint16_t* vc, uint16_t* out, int H,
                                      int Hkv, int64_t pos0, int64_t Lmax, float scale, int64_t window, int64_t sinks,
                                      cudaStream_t s);
cudaError_t launch_gqa_attention_window(const uint16_t* q, const uint16_t* kc, const uint16_t* vc, uint16_t* out,
                                        int64_t M, int H, int Hkv, int64_t pos0, int64_t Lmax, float scale,
                                        int64_t window, int64_t sinks, cudaStream_t s);
uint32_t attn_take_status();

// The 4-bit cache: rows of D values as D / 2 bytes (q4) and D / 32 pairs of fp16
// (dm), [H_kv][Lmax] of them.  Arguments validated.
struct Q4Cache {
  const uint8_t *k_q4, *v_q4;
  const uint16_t *k_dm, *v_dm;
};
// fp16 rows k_out[g][r] and, unless v_out is null (c.v_q4 and c.v_dm are not read then),
// v_out[g][r]: row r is position r where r < sinks, else r + gap.
cudaError_t launch_dequant_kv_q4(const Q4Cache& c, uint16_t* k_out, uint16_t* v_out, int Hkv, int D, int64_t Lmax,
                                 int64_t rows, int64_t sinks, int64_t gap, cudaStream_t s);
// qk_gqa_attention_q4: few tokens by the decode kernel, others through the
// scratch (attn_q4_scratch bytes).
int64_t attn_q4_scratch(int64_t M, int H, int Hkv, int64_t pos0, int64_t window, int64_t sinks);
cudaError_t launch_gqa_attention_q4(const uint16_t* q, const Q4Cache& c, uint16_t* out, int64_t M, int H, int Hkv,
                                    int64_t pos0, int64_t Lmax, float scale, int64_t window, int64_t sinks,
                                    void* scratch, cudaStream_t s);
uint32_t attn_win_take_status();

// A kernel whose single bounded wait can never complete (see qk_debug_wait_timeout).
cudaError_t launch_wait_probe(uint64_t limit_ns, cudaStream_t s);

// Largest M the GEMV handles (M = 1 in the decode layout, 2..8 with the
// tokens in the MMA columns); larger M goes to the tensor-core GEMM, which
// measured faster there on GB300 (Q4_K 3072 x 3072 at M = 16: 15 vs 24 us).
constexpr int kMaxGemvM = 8;
int gemv_max_m();
// The kernel's token-slot count for M tokens (1 or 8): problems share a
// launch only with problems of the same count.
int gemv_slots(int64_t M);

// One problem of a grouped GEMV launch.  w1 != null makes it the fused
// gate/up + SwiGLU problem (w0 = gate, w1 = up, y fp16), else y is fp32.
constexpr int kMaxGemvProbs = 8;
struct GemvDesc {
  QType qtype;
  const void* w0;
  const void* w1;
  const uint16_t* x;
  void* y;
  int64_t M, N, K;
  const uint16_t* gamma;  // RMSNorm prologue over x (fp16 gamma[K]), or null
  float eps;
  bool q8x = false;       // x quantized to int8 per block of 32 (one token, no gamma)
  const float* xd = nullptr;  // q8x with x given in int8: x points at the values, xd at their K / 32 scales
};
cudaError_t launch_gemv_batch(const GemvDesc* d, int count, cudaStream_t s);

// Whether one grouped GEMV launch can run these problems: each problem's own
// plan (its x table and at least two weight stages) must fit in shared memory
// and all must have the same token-slot count.  Host only (no CUDA call).
// Problems that do not fit run on the GEMM.
bool gemv_plan_fits(const GemvDesc* d, int count);

}  // namespace qk
