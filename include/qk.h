/*
 * qk.h -- C ABI of libqk: fused dequantize-and-multiply of GGUF Q4_K / Q6_K
 * weights with fp16 activations on NVIDIA GB300 (sm_103a).
 *
 * What the library computes (DAMASCUS project overview, "[01] the thesis",
 * "[04] one decode step"; "Building DAMASCUS", "Read the model, then
 * reproduce its operations" and "Prefill and decode need different
 * performance questions"):
 *   every linear layer of a Llama-3.2-3B decoder (QKV, O, SwiGLU gate/up,
 *   down, tied LM head) as y = x . W^T with W stored as quantized Q4_K / Q6_K
 *   super-blocks and dequantized on the fly; decode is the M = 1 case (a
 *   bandwidth-bound GEMV), prefill the M > 1 case (a compute-bound GEMM).
 *
 * Block formats (public GGUF definitions; the pages name them but do not print
 * their layout):
 *   Q4_K, 144 bytes per 256 weights: fp16 d, fp16 dmin, 12 bytes of packed
 *     6-bit scales/mins for 8 sub-blocks of 32, 128 bytes of 4-bit quants;
 *     w = (d * sc) * q - (dmin * m).
 *   Q6_K, 210 bytes per 256 weights: 128 bytes low 4 bits, 64 bytes high 2
 *     bits, 16 int8 scales (one per 16 weights), fp16 d;
 *     w = (d * sc) * (q - 32).
 *
 * Conventions for every entry point:
 *   - Weights W: N rows of K/256 consecutive blocks (row n = output feature n),
 *     rows packed back to back (row stride = K/256 * block bytes).
 *   - x: [M][K] fp16 (IEEE binary16 bit patterns), row-major, dense.
 *   - y: [M][N] row-major, dense (fp32, or fp16 for the SwiGLU entry point).
 *   - All pointers are DEVICE pointers of the current CUDA device (or mapped
 *     host memory the device can read), 16-byte aligned.  The caller owns every
 *     buffer; the library allocates no device memory on any call.
 *   - K must be a positive multiple of 256 and N, K below 2^31; M is at most
 *     8,388,480 (65535 token tiles of 128).  M = 0 or N = 0 is a no-op.
 *   - y must not overlap x or the weights.
 *   - Work is enqueued asynchronously on `stream` (NULL = legacy default
 *     stream).  The return value reports argument and launch errors only; a
 *     kernel that gives up on a bounded wait sets a device flag that
 *     qk_get_device_status() reports.
 *   - No entry point aborts, exits or traps.
 *   - Results are deterministic: the same inputs give bit-identical outputs.
 */
#ifndef QK_H
#define QK_H

#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef int qk_status;

#define QK_OK 0
#define QK_ERR_NULL (-1)               /* a required pointer is NULL */
#define QK_ERR_ALIGN (-2)              /* a pointer is not 16-byte aligned */
#define QK_ERR_SHAPE (-3)              /* K % 256 != 0, a negative size, or a size beyond the limits */
#define QK_ERR_CUDA (-4)               /* a CUDA runtime call or kernel launch failed */
#define QK_ERR_TIMEOUT (-5)            /* a kernel gave up on a bounded wait (see qk_get_device_status) */
#define QK_ERR_UNSUPPORTED_DEVICE (-6) /* the current device is not an sm_103 GPU */
#define QK_ERR_ALIAS (-7)              /* the output overlaps an input */
#define QK_ERR_POINTER (-8)            /* a pointer is not accessible from the current device */
#define QK_ERR_SCRATCH (-9)            /* the built-in scratch of qk_rmsnorm_matmul_batch_static is too small */
#define QK_ERR_BAD_COPY (-10)          /* debug builds (QK_DEBUG) only: a kernel skipped a bulk or tensor copy
                                          whose addresses, size or shared-memory extent failed its check */

/* A cudaStream_t, spelled without CUDA headers. */
typedef struct CUstream_st *qk_stream_t;

/*
 * Dequantize n_blocks consecutive Q4_K blocks (144 B each) into n_blocks*256
 * fp32 weights, out[256*b + i] = weight i of block b.  Bit-exact with the
 * fp32 expression fp32(fp32(d)*sc)*q - fp32(fp32(dmin)*m) evaluated left to
 * right with round-to-nearest and no fused multiply-add ("Building DAMASCUS",
 * "Read the model, then reproduce its operations": the dequantizers are the
 * first correctness boundary).  n_blocks = 0 is a no-op.
 */
qk_status qk_dequant_q4k(const void *blocks, int64_t n_blocks, float *out, qk_stream_t stream);

/* As qk_dequant_q4k for Q6_K blocks (210 B each): w = fp32(fp32(d)*sc)*(q-32). */
qk_status qk_dequant_q6k(const void *blocks, int64_t n_blocks, float *out, qk_stream_t stream);

/*
 * Number range of the two paths.  The GEMV (M <= 8) applies the block scales
 * in fp32.  The tensor-core GEMM forms every weight in fp16: fp16(d*sc),
 * fp16(dmin*m) and fp16(q*d*sc - dmin*m), each rounded from fp32; a block
 * whose |d*sc*q| or |dmin*m| exceeds 65504 gives +-inf weights there (the
 * synthetic and real Llama scales are near 1e-4).  A non-finite d or dmin
 * makes its row's outputs non-finite on every path, as in the fp32 definition.
 */

/*
 * y[m][n] = sum_k x[m][k] * w[n][k] for Q4_K weights W (N x K), fp16 x, fp32 y
 * (DAMASCUS project overview, "[01] the thesis" / "[04] one decode step";
 * "Building DAMASCUS", "Prefill and decode need different performance
 * questions").  M <= 8 runs the GEMV (products of the integer quants with
 * fp16 x are exact, sums fp32, block scales applied per sub-block in fp32)
 * where its shared-memory plan fits (see qk_uses_gemv: the model's K = 3072
 * and K = 8192 up to M = 8); larger M, and problems the GEMV cannot
 * stage, run the tensor-core GEMM (weights dequantized to fp16 in
 * shared or tensor memory, never written to device memory; fp32 accumulation
 * in tensor memory),
 * the overview's prefill plan in which dequantized weights feed the matrix
 * unit directly and no fp16 copy of them is stored.  The two paths agree within rounding; results are not
 * bit-identical across M.  Single-tensor GEMMs keep the dequantized tiles in
 * tensor memory where they fit; QK_A_TMEM=0 in the environment (read once per
 * process) selects shared memory instead, with the same results within
 * rounding.
 */
qk_status qk_matmul_q4k(const void *blocks, const uint16_t *x_f16, float *y, int64_t M, int64_t N, int64_t K,
                        qk_stream_t stream);

/* As qk_matmul_q4k for Q6_K weights. */
qk_status qk_matmul_q6k(const void *blocks, const uint16_t *x_f16, float *y, int64_t M, int64_t N, int64_t K,
                        qk_stream_t stream);

/*
 * Fused SwiGLU feed-forward input projection (DAMASCUS project overview,
 * "[04] one decode step" and "[06] the target": FFN = SwiGLU):
 *   g = x . Wg^T, u = x . Wu^T (both N_ff x K, Q4_K), fp32 accumulation,
 *   y[m][n] = fp16( g / (1 + exp(-g)) * u ), y is [M][N_ff] fp16.
 * Gate and up weights are two separate Q4_K tensors of the same shape.  The
 * tensor-core path (M > 1) evaluates the sigmoid as 0.5 + 0.5 * tanh(g / 2)
 * with the hardware tanh approximation (relative error about 2^-11); the
 * result agrees with the definition within the fp16 output's rounding plus
 * that error.
 */
qk_status qk_gateup_swiglu_q4k(const void *gate_blocks, const void *up_blocks, const uint16_t *x_f16,
                               uint16_t *y_f16, int64_t M, int64_t N_ff, int64_t K, qk_stream_t stream);

/* Weight formats for qk_matmul_desc.qtype. */
#define QK_Q4_K 0
#define QK_Q6_K 1

/*
 * One problem of a grouped call.  up_blocks == NULL: y[M][N] (fp32) = x . W^T
 * with W in format `qtype`.  up_blocks != NULL: the fused gate/up + SwiGLU of
 * qk_gateup_swiglu_q4k (qtype must be QK_Q4_K, blocks = gate, y fp16).
 */
typedef struct qk_matmul_desc {
  int qtype;
  const void *blocks;
  const void *up_blocks;
  const uint16_t *x_f16;
  void *y;
  int64_t M, N, K;
} qk_matmul_desc;

/*
 * Run `count` independent problems (DAMASCUS project overview, "[04] one
 * decode step": the QKV projections share x, gate and up share x, and every
 * decode-step linear is an M = 1 GEMV).  Problems the GEMV runs (M <= 8)
 * share launches, up to 8 per launch, with the problems of the same
 * token-slot class (M = 1; 2..8), so small GEMVs stream their weights
 * concurrently; each keeps its own shared-memory plan and split over warps.
 * Other problems run as in qk_matmul_q4k / qk_matmul_q6k /
 * qk_gateup_swiglu_q4k.  Each entry obeys the rules of its single-problem
 * entry point; in addition no y may overlap any input or output of another
 * entry.  count = 0 is a no-op.  Results are bit-identical to calling the
 * single-problem entry points one by one.
 */
qk_status qk_matmul_batch(const qk_matmul_desc *descs, int count, qk_stream_t stream);

/*
 * int8 activations (the paper has no integer-activation variant: this is a
 * trade of accuracy for arithmetic this library offers beside the fp16
 * path).  Decode only (M = 0 or 1).  Each token's x is quantized per block of
 * 32 to int8 with one fp32 scale: d = amax / 127, q = round(x / d) (IEEE fp32
 * division, ties away from zero; d = 0 gives q = 0); y = sum_k d q w with the
 * products done as integer dot products and the block scales applied in fp32.
 * The result differs from the fp16 path by the quantization of x: per output
 * at most sum over 32-blocks of (d / 2) * sum |w| (finite x).  Problems whose K
 * the decode GEMV cannot stage are refused with QK_ERR_SHAPE (there is no
 * other int8 path).  Descriptors and rules as in qk_matmul_batch (up_blocks:
 * the fused gate/up + SwiGLU); M > 1 is QK_ERR_SHAPE.
 */
qk_status qk_matmul_batch_q8x(const qk_matmul_desc *descs, int count, qk_stream_t stream);
qk_status qk_matmul_q8x_q4k(const void *blocks, const uint16_t *x_f16, float *y, int64_t M, int64_t N, int64_t K,
                            qk_stream_t stream);
qk_status qk_matmul_q8x_q6k(const void *blocks, const uint16_t *x_f16, float *y, int64_t M, int64_t N, int64_t K,
                            qk_stream_t stream);

/*
 * RMSNorm in front of the linears (DAMASCUS project overview, "[04] one decode
 * step": an RMSNorm comes before the QKV projections and before the SwiGLU
 * FFN; "Building DAMASCUS", "Read the model, then reproduce its operations").
 * Every problem's x is replaced by
 *   xhat[m][k] = fp16( x[m][k] / sqrt(mean_k x[m][k]^2 + eps) * gamma[k] )
 * (sum of squares, scale and products in fp32; gamma is fp16[K], the same K
 * for every problem of the call; eps finite and >= 0) and the problems then
 * run as in qk_matmul_batch.  Problems the GEMV runs (M <= 8 where its plan
 * fits with gamma beside x; qk_uses_gemv answers for no norm, and some K fit
 * there alone) normalize inside its x staging: no extra pass, no scratch.
 * Problems the tensor-core GEMM runs first have their xhat written to
 * `scratch`, a caller-owned device buffer of at least qk_rmsnorm_scratch_bytes
 * (the largest M * K * 2 over those problems; NULL is allowed when no problem
 * needs it); problems run in order on `stream` and share it.  scratch must
 * not overlap gamma or any input or output; the library cannot check its
 * size.  Returns QK_ERR_NULL (gamma, or scratch when needed), QK_ERR_ALIGN,
 * QK_ERR_SHAPE (eps negative or not finite, problems of different K), and the
 * codes of qk_matmul_batch.
 */
qk_status qk_rmsnorm_matmul_batch(const qk_matmul_desc *descs, int count, const uint16_t *gamma_f16, float eps,
                                  void *scratch, qk_stream_t stream);

/* One problem of qk_rmsnorm_matmul_batch: y = (RMSNorm(x) * gamma) . W^T, Q4_K or Q6_K weights. */
qk_status qk_rmsnorm_matmul_q4k(const void *blocks, const uint16_t *x_f16, const uint16_t *gamma_f16, float eps,
                                void *scratch, float *y, int64_t M, int64_t N, int64_t K, qk_stream_t stream);
qk_status qk_rmsnorm_matmul_q6k(const void *blocks, const uint16_t *x_f16, const uint16_t *gamma_f16, float eps,
                                void *scratch, float *y, int64_t M, int64_t N, int64_t K, qk_stream_t stream);

/* The fused gate/up + SwiGLU of qk_gateup_swiglu_q4k over RMSNorm(x) * gamma. */
qk_status qk_rmsnorm_gateup_swiglu_q4k(const void *gate_blocks, const void *up_blocks, const uint16_t *x_f16,
                                       const uint16_t *gamma_f16, float eps, void *scratch, uint16_t *y_f16,
                                       int64_t M, int64_t N_ff, int64_t K, qk_stream_t stream);

/*
 * qk_rmsnorm_matmul_batch without a scratch argument, for callers that cannot
 * allocate device memory: code running while a CUDA graph is being captured
 * (an allocation there is not recorded into the graph), callers inside a
 * framework whose memory pool owns the GPU's memory, and real-time loops that
 * allocate nothing after start-up because cudaMalloc can block and
 * synchronise the device.  The paper has no counterpart of this entry point:
 * it is a convenience of this library, not part of the method.
 *
 * The normalized activations of problems the tensor-core GEMM runs go to a
 * fixed 8 MiB array inside the library instead (every GPU that loads the
 * library holds it until the process exits): the largest M * K over those
 * problems must be at most 4,194,304 (M * K * 2 bytes <= 8 MiB), else the call
 * returns QK_ERR_SCRATCH and enqueues nothing.  The call allocates nothing and
 * calls no allocating routine.  Every call shares the array and it keeps the
 * last call's contents (each call overwrites what it reads), so calls whose
 * work may overlap on the GPU -- on different streams, or from several host
 * threads -- race on it; serialise them.  The first call on a device that
 * needs the array looks up its device address (cudaGetSymbolAddress, with
 * that device current) and keeps it; make that first call before capturing
 * any stream.  Otherwise as qk_rmsnorm_matmul_batch.
 */
qk_status qk_rmsnorm_matmul_batch_static(const qk_matmul_desc *descs, int count, const uint16_t *gamma_f16, float eps,
                                         qk_stream_t stream);

/*
 * Host-only query: bytes of scratch an M-token problem of this format and K
 * needs under qk_rmsnorm_matmul_batch (0 when the GEMV fuses the norm, else
 * M * K * 2), or -1 for invalid arguments.
 */
int64_t qk_rmsnorm_scratch_bytes(int qtype, int gateup, int64_t M, int64_t K);

/*
 * int8 activations that are quantized already (by qk_add_rmsnorm_q8, say):
 * one token's x as K int8 values x_q8 and K / 32 fp32 scales x_d,
 *   y[n] = sum_k x_d[k / 32] x_q8[k] w[n][k],
 * with the arithmetic of qk_matmul_batch_q8x: for the x_q8 and x_d that
 * qk_matmul_batch_q8x would compute from an fp16 x the results are
 * bit-identical.  up_blocks != NULL: the fused gate/up + SwiGLU, y fp16.
 * M must be 0 or 1 and K one that the decode GEMV can stage, as there; x_q8
 * and x_d are 16-byte aligned.  Rules and errors as in qk_matmul_batch_q8x.
 */
typedef struct qk_matmul_q8_desc {
  int qtype;
  const void *blocks;
  const void *up_blocks;
  const int8_t *x_q8;
  const float *x_d;
  void *y;
  int64_t M, N, K;
} qk_matmul_q8_desc;

qk_status qk_matmul_batch_q8(const qk_matmul_q8_desc *descs, int count, qk_stream_t stream);

/* Element types of a residual stream. */
#define QK_F16 0
#define QK_F32 1

/*
 * Residual addition and RMSNorm between two linears (DAMASCUS project
 * overview, "[04] one decode step": residual, then RMSNorm, before the QKV
 * projections and before the FFN).  For each of M rows of K values
 *   h = residual + delta                              (fp32 sum)
 *   residual_out = h                                  (rounded to the residual's type)
 *   xhat = fp16( h / sqrt(mean_k h^2 + eps) * gamma ) (fp32 arithmetic on the unrounded h)
 * residual is fp16 or fp32 (residual_type QK_F16 / QK_F32), delta the fp32
 * output of a linear, or NULL for h = residual; gamma fp16[K].  residual_out
 * may be the residual itself (in place) or NULL (not wanted); xhat feeds the
 * linears.  K is a positive multiple of 8 below 2^31, M at most 2^31 - 1.
 * Outputs may not overlap each other or an input, save residual_out ==
 * residual.  h^2 must stay within fp32.
 * qk_add_rmsnorm_q8 writes the activations in int8 instead, quantized from
 * the fp16 xhat as the q8x matmuls quantize (per 32 values d = amax / 127,
 * q = round(xhat / d), ties away from zero, d = 0 gives q = 0; finite xhat):
 * xq int8 [M][K] and xd fp32 [M][K / 32], one row of which is the x of
 * qk_matmul_batch_q8.  K is a multiple of 32 there.
 * How many threads share a row follows M and the device, so the last bit of a
 * row can differ between calls of different M; the same call repeats its bits.
 * qk_matmul_batch_q8 takes one row of qk_add_rmsnorm_q8's output a call.
 * M = 0 is a no-op.
 */
qk_status qk_add_rmsnorm(const void *residual, int residual_type, const float *delta, const uint16_t *gamma_f16,
                         float eps, void *residual_out, uint16_t *xhat_f16, int64_t M, int64_t K, qk_stream_t stream);
qk_status qk_add_rmsnorm_q8(const void *residual, int residual_type, const float *delta, const uint16_t *gamma_f16,
                            float eps, void *residual_out, int8_t *xq, float *xd, int64_t M, int64_t K,
                            qk_stream_t stream);

/* Which dimensions of a head turn together: (2i, 2i + 1) or (i, i + n_rot / 2). */
#define QK_ROPE_INTERLEAVED 0
#define QK_ROPE_HALF 1

/*
 * Rotary positions, and the new rows of the KV cache ("[04] one decode step":
 * RoPE between the QKV projections and the attention over the cache; "[06] the
 * target": theta = 500000).  From the fp32 outputs q [M][H][D], k and v
 * [M][H_kv][D] of the QKV projections: q_f16 [M][H][D], and rows pos0 ..
 * pos0 + M - 1 of k_cache and v_cache [H_kv][L_max][D], all fp16; other cache
 * rows are left as they were.  Token i is at position p = pos0 + i; pair j of
 * the first n_rot dimensions of every q and k head turns by p * inv_freq[j]:
 *   (a, b) -> magnitude * (a cos - b sin, b cos + a sin);
 * the other dimensions, and v, are only rounded.  inv_freq: n_rot / 2 doubles
 * in device memory (qk_rope_inv_freq makes them), so that the angle of a far
 * position keeps its fraction of a turn.  D is a multiple of 8, at most 512;
 * n_rot even, 0 .. D (0: nothing turns, inv_freq may be NULL); pos0 + M <=
 * L_max < 2^31; H and H_kv at most 1024; magnitude finite.  No two buffers
 * may overlap.  M = 0 is a no-op.
 */
qk_status qk_rope_kv_append(const float *q, const float *k, const float *v, const double *inv_freq, uint16_t *q_f16,
                            uint16_t *k_cache, uint16_t *v_cache, int64_t M, int64_t H, int64_t H_kv, int64_t D,
                            int64_t n_rot, int64_t pos0, int64_t L_max, int layout, float magnitude,
                            qk_stream_t stream);

/*
 * qk_rope_kv_append with an RMSNorm of every query and key head in front, for
 * models that normalize them: a head's D values x become
 *   x / sqrt(mean x^2 + eps) * gamma      (fp32; before the rotation)
 * with q_gamma_f16 for the query heads and k_gamma_f16 for the key heads, fp16[D]
 * each; where a gamma is NULL its heads are not normalized.  v never is.  eps is
 * finite and >= 0, and x^2 must stay within fp32.  The rest as in
 * qk_rope_kv_append; M is below 2^31.
 * qk_norm_rope_kv_append_q4 writes the new rows into a cache held in 4 bits,
 * k_q4 and v_q4 [H_kv][L_max][D / 2] bytes with k_dm and v_dm
 * [H_kv][L_max][D / 32][2] fp16, D a multiple of 32.  Each 32 values x of a row
 * are a group, held as v = d q + m:
 *   m = fp16(min x),  d = fp16(max(max x - m, 0) / 15),
 *   q = the nearest of 0 .. 15 to (x - m) / d (ties to even; 0 where d = 0),
 * from the fp32 values and in fp32.  Byte j of a group has the q of value 2 j in
 * its low and of 2 j + 1 in its high half; dm has d, then m.  A group with a value
 * that is not finite or not below 65520 in size (fp16 has none for it), or with d
 * above 4366 (values more than about 65490 apart: 15 d would not be a finite fp16
 * number), is stored as NaN (d and m).  Where 15 d + m would be 65520 or more, as d
 * was rounded up, d is the next fp16 number below: d q + m is a finite fp16 number
 * for every q of a group that is not NaN.
 */
qk_status qk_norm_rope_kv_append(const float *q, const float *k, const float *v, const uint16_t *q_gamma_f16,
                                 const uint16_t *k_gamma_f16, float eps, const double *inv_freq, uint16_t *q_f16,
                                 uint16_t *k_cache, uint16_t *v_cache, int64_t M, int64_t H, int64_t H_kv, int64_t D,
                                 int64_t n_rot, int64_t pos0, int64_t L_max, int layout, float magnitude,
                                 qk_stream_t stream);
qk_status qk_norm_rope_kv_append_q4(const float *q, const float *k, const float *v, const uint16_t *q_gamma_f16,
                                    const uint16_t *k_gamma_f16, float eps, const double *inv_freq, uint16_t *q_f16,
                                    uint8_t *k_q4, uint16_t *k_dm, uint8_t *v_q4, uint16_t *v_dm, int64_t M, int64_t H,
                                    int64_t H_kv, int64_t D, int64_t n_rot, int64_t pos0, int64_t L_max, int layout,
                                    float magnitude, qk_stream_t stream);

/*
 * Rows pos0 .. pos0 + M - 1 of one tensor of a 4-bit cache as fp16:
 * out_f16[g][r] = fp16(d q + m) (one rounding) of position pos0 + r, [H_kv][M][D].
 * D is a multiple of 32, at most 512; pos0 + M <= L_max < 2^31; H_kv at most 1024.
 */
qk_status qk_dequant_kv_q4(const uint8_t *q4, const uint16_t *dm, uint16_t *out_f16, int64_t H_kv, int64_t D,
                           int64_t pos0, int64_t M, int64_t L_max, qk_stream_t stream);

/*
 * Host-only: the rotation frequencies, in radians per position, into
 * out[0 .. n_rot / 2 - 1] (host memory; the caller copies them to the device).
 *   f_i = theta^(-2 i / n_rot) / freq_factors[i]  (freq_factors NULL: 1),
 * then, by `scaling`:
 *   QK_ROPE_SCALE_NONE    f_i
 *   QK_ROPE_SCALE_LINEAR  f_i / factor
 *   QK_ROPE_SCALE_BANDED  (1 - g) f_i / factor + g f_i, with
 *     g = clamp((t_i - low_turns) / (high_turns - low_turns), 0, 1) and
 *     t_i = original_len f_i / (2 pi), the turns of pair i over the context the
 *     model was trained with: pairs of many turns keep their frequency, pairs
 *     of few are slowed by `factor`.  (YaRN's ramp, Peng et al. 2023, has
 *     low_turns 1 and high_turns 32, and a magnitude of 0.1 ln(factor) + 1 for
 *     qk_rope_kv_append; Llama-3.2's own scaling low_turns 1 and high_turns 4.)
 * theta and factor must be positive and finite, freq_factors positive and
 * finite, high_turns > low_turns >= 0 and original_len > 0 where they are
 * used, n_rot even and 0 .. 512; else QK_ERR_SHAPE.
 */
#define QK_ROPE_SCALE_NONE 0
#define QK_ROPE_SCALE_LINEAR 1
#define QK_ROPE_SCALE_BANDED 2
typedef struct qk_rope_config {
  double theta;
  int scaling;
  double factor;
  double low_turns, high_turns;
  int64_t original_len;
  const float *freq_factors; /* host memory, n_rot / 2 values, or NULL */
} qk_rope_config;

qk_status qk_rope_inv_freq(const qk_rope_config *config, int64_t n_rot, double *out);

/*
 * Grouped-query attention over a KV cache (DAMASCUS project overview, "[02]
 * the pipeline", compartment 06: a decoder layer is GQA with a KV cache; "[04]
 * one decode step": after the QKV projections and RoPE, attention over the
 * cache).  The pages print no formula; this is scaled dot-product attention:
 * for query i (0 <= i < M) at position pos0 + i and query head h, with
 * g = h / (H / H_kv) its key/value head,
 *   s_j = scale * sum_d q[i][h][d] * k_cache[g][j][d]   for j = 0 .. pos0 + i,
 *   out[i][h][d] = sum_j softmax(s)_j * v_cache[g][j][d].
 * q_f16: [M][H][D] fp16 (RoPE already applied); k_cache, v_cache: [H_kv][L_max][D]
 * fp16, positions 0 .. pos0 + M - 1 filled (those of the M queries included);
 * out: [M][H][D] fp32.  D must be 128, H a multiple of H_kv with H / H_kv <= 8,
 * pos0 + M <= L_max; all pointers device memory, 16-byte aligned; out may not
 * overlap an input.  M = 1 (a decode step) splits the cache over a cluster of
 * up to 8 CTAs per key/value head; M >= 2 (prefill, or a chunk of it after
 * pos0 cached positions) runs causal 128-query blocks on tcgen05.  Both score
 * on the tensor cores (fp16 operands, fp32 sums) and round the softmax weights
 * to fp16 for the P.V product (weights below 2^-25 of the largest count in the
 * sum alone): the result is within about (2^-11 + n 2^-25) * max|v| of the exact
 * value for n visible positions, 2^-10 up to 2^14 of them; in decode n is what
 * one warp takes of them, about 1 / 64 from 2048 positions on.  M = 0 is a
 * no-op.  Errors: QK_ERR_SHAPE, QK_ERR_NULL, QK_ERR_ALIGN, QK_ERR_ALIAS,
 * QK_ERR_POINTER, QK_ERR_UNSUPPORTED_DEVICE before anything is enqueued;
 * QK_ERR_CUDA if the launch fails.
 */
qk_status qk_gqa_attention(const uint16_t *q_f16, const uint16_t *k_cache, const uint16_t *v_cache, float *out,
                           int64_t M, int64_t H, int64_t H_kv, int64_t D, int64_t pos0, int64_t L_max, float scale,
                           qk_stream_t stream);

/*
 * qk_gqa_attention with a sliding window and sinks, and an fp16 output that
 * the O projection reads as it is: query i at position p = pos0 + i sees
 * position j <= p when j > p - window or j < sinks (the window's last `window`
 * positions, itself included, and the first `sinks` of the sequence).  window
 * and sinks are >= 0; a window of at least pos0 + M is plain causal attention,
 * and a query that sees nothing (window = sinks = 0) gives zeros.  Only the
 * rows of the caches that some query of the call sees are used: rows between
 * the sinks and the first query's window, and rows past the last query, may
 * hold anything.  What a row holds, NaN and infinities included, reaches the
 * queries that see it and no other (an infinite value whose weight rounds to 0
 * arrives as NaN; with scale 0, M >= 2, an infinite score is infinite still).
 * Non-finite results are slow for M >= 2: each such row and head is computed
 * again by one warp, so an infinite value that a whole chunk sees costs 100 to
 * 1000 times the chunk's time (4095 queries, 24 heads, window 2048: 0.11 ms ->
 * 39 ms).  scale is finite, and scale * log2(e) * q . k must stay within fp32
 * for finite q and k.  Other arguments, limits and errors as in
 * qk_gqa_attention; out: [M][H][D] fp16, within about 2^-10 * max|v| of the
 * exact value plus its own rounding where a query sees 2^20 positions at most
 * (in prefill weights down to 2^-32 of the largest count; decode as in
 * qk_gqa_attention).  Finite values give finite results.  How a chunk's work is
 * shared among CTAs follows M, so a query's last bits can differ between chunks
 * of different sizes; the same call repeats its bits.
 */
qk_status qk_gqa_attention_window(const uint16_t *q_f16, const uint16_t *k_cache, const uint16_t *v_cache,
                                  uint16_t *out_f16, int64_t M, int64_t H, int64_t H_kv, int64_t D, int64_t pos0,
                                  int64_t L_max, float scale, int64_t window, int64_t sinks, qk_stream_t stream);

/*
 * qk_gqa_attention_window over a cache held in 4 bits (the layout of
 * qk_norm_rope_kv_append_q4; d q + m and 15 d must be finite fp16 numbers, or d
 * or m NaN).  Up to 32 columns, M * H / H_kv (a decode step, or a few drafted
 * tokens), read the 4-bit rows directly: over a cluster of CTAs per key/value
 * head, or, from 65536 positions of all key/value heads on, over all SMs, joined
 * by a second kernel through `scratch`.  More tokens have the rows that their
 * queries see written to `scratch` as fp16 first (512 bytes a position and
 * key/value head).  scratch is a caller-owned device buffer of at least
 * qk_gqa_attention_q4_scratch_bytes, NULL where that is 0; what it holds before
 * and after is of no account.  Calls that may overlap on the GPU need a scratch
 * each, captured graphs included.  The library cannot check its size.  pos0 + M
 * is below 2^30.  Window, sinks, rows that no query sees, other limits, accuracy,
 * non-finite rows (not slow for few tokens) and errors as in
 * qk_gqa_attention_window.  Measured of random rows, as the 2-norm of the error over
 * that of the output (rounding exact outputs to fp16 leaves 2.1e-4): few tokens,
 * whose weights and d (q - 8) of V are rounded to fp16, 2.8e-4 after 500 positions and
 * 3.3e-4 after 65536; more tokens, whose rows are rounded instead, 5.8e-4.  The same
 * query may therefore differ in its last bits with the number of tokens in its call.
 */
qk_status qk_gqa_attention_q4(const uint16_t *q_f16, const uint8_t *k_q4, const uint16_t *k_dm, const uint8_t *v_q4,
                              const uint16_t *v_dm, uint16_t *out_f16, int64_t M, int64_t H, int64_t H_kv, int64_t D,
                              int64_t pos0, int64_t L_max, float scale, int64_t window, int64_t sinks, void *scratch,
                              qk_stream_t stream);

/* Host-only query: bytes of scratch that such a call needs (0: none), or -1 for invalid arguments. */
int64_t qk_gqa_attention_q4_scratch_bytes(int64_t M, int64_t H, int64_t H_kv, int64_t D, int64_t pos0, int64_t window,
                                          int64_t sinks);

/*
 * Log probabilities from the LM head's logits (the pages' "[02] the pipeline",
 * compartments 06 and 07: the tied LM head's logits go to the sampler).  For
 * each row m of logits fp32 [M][V], with lse = log sum_v exp(logits[m][v]):
 *   logprob[m]          = logits[m][tokens[m]] - lse
 *   entropy[m]          = lse - sum_v p_v logits[m][v],  p_v = exp(logits[m][v] - lse)
 *   top_ids[m][i]       = the token of the i-th largest logit, i = 0 .. top_n - 1
 *   top_logprobs[m][i]  = its log probability.
 * Equal logits order by the lower token.  -inf logits (banned tokens) have
 * probability 0 and add nothing to the entropy; NaN logits order below -inf.
 * A row that holds NaN or +inf, or nothing but -inf, has NaN log probabilities
 * and entropy; its top_ids are still the order above.  A token outside 0 ..
 * V - 1 (padding) gives a NaN logprob.  logprob and tokens go together
 * (both NULL: not wanted), so do top_ids and top_logprobs (top_n = 0); entropy
 * may be NULL.  0 <= top_n <= 32 and top_n <= V; V below 2^31, M at most
 * 2^31 - 1.  Rows need not be 16-byte aligned (any V), the buffers do.  No
 * output may overlap another or an input.  How many CTAs share a row follows M
 * and the device, so the last bits of its sums can differ between calls of
 * different M; the same call repeats its bits, and the ids never differ.  M = 0
 * is a no-op; V = 0 is QK_ERR_SHAPE.
 */
qk_status qk_logprobs(const float *logits, const int32_t *tokens, float *logprob, float *entropy, int top_n,
                      int32_t *top_ids, float *top_logprobs, int64_t M, int64_t V, qk_stream_t stream);

/*
 * A token from each row of logits fp32 [M][V] (the pages' "[02] the pipeline",
 * compartment 07: the sampler) and a given uniform random number u[m] in 0 .. 1.
 * With a row's tokens in descending order of their logits x (equal ones by the
 * lower token; -inf, banned tokens, never count), w = exp((x - max x) / temperature)
 * and C(n) the sum of the first n weights, the kept tokens are the first n, the
 * least of
 *   top_k (0: all of them),
 *   the first n with C(n) >= top_p C(top_k)   (top_p 1: all),
 *   the number of tokens with w >= min_p      (min_p 0: all),
 * and
 *   token[m]   = the first in that order whose C exceeds u[m] C(n),
 *   logprob[m] = log of its share w / C(n) of the kept weights (may be NULL),
 *   kept[m]    = n (may be NULL).
 * temperature 0 gives the first token in the order, a logprob of 0 and kept 1.  A
 * row that holds NaN or +inf, or nothing but -inf, gives token -1, a NaN logprob
 * and kept 0.  u below 0 or NaN counts as 0, u of 1 or more as the largest fp32
 * number below 1.  A weight is within 2^-36 of itself.  An addition rounds off at most
 * 3 2^-48 of its thread's sum, which starts at the largest weight, and what the threads
 * hold is rounded to 2^-44 of that: together less than 2^-28 of the sum (2^-27 for V above
 * 2^17).  A token therefore follows from the definition rather than from the order of a
 * sum, but where a border lies closer than that to a decision.
 * How many CTAs share a row follows M and the device, and with it the sums' last
 * bits; the same call repeats its bits.  temperature is 0 or 1e-6 .. 1e6, top_p
 * 0 .. 1, min_p 0 or 1e-12 .. 1, V at most 524288, M at most 2^31 - 1.  Rows need
 * not be 16-byte aligned (any V), the buffers do.  No output may overlap another or
 * an input.  Thousands of equal logits around the last kept token, or around the
 * chosen one (logits of few bits), make a row slow: it is then searched by one CTA, a
 * pass for every bit.  Up to 8 ms were measured for a row of 128256 logits and 34 ms
 * for one of 524288; 18 and 80 ms for calls of 300 such rows.  M = 0 is a no-op;
 * V = 0 is QK_ERR_SHAPE.
 */
qk_status qk_sample(const float *logits, const float *u, int32_t *token, float *logprob, int32_t *kept, int64_t M,
                    int64_t V, float temperature, int top_k, float top_p, float min_p, qk_stream_t stream);

/*
 * Synchronise `stream`, then report and clear the device-side status flags
 * that the library's kernels set when a bounded wait expires.  Returns QK_OK,
 * QK_ERR_TIMEOUT, or QK_ERR_CUDA if the synchronisation itself failed.  A
 * library built with -DQK_DEBUG also checks each bulk and tensor copy before
 * issuing it (shared-memory destination and mbarrier aligned and inside the
 * CTA's shared memory; source and size of a plain bulk copy 16-byte aligned)
 * and returns QK_ERR_BAD_COPY, ahead of QK_ERR_TIMEOUT, when one failed.
 * The flags belong to the current device, not to a stream: every stream of
 * the process on that device sets the same flags.  A timeout raised by a
 * kernel on another stream that has already finished is therefore reported
 * (and cleared) by whichever call reads the flags first, and a kernel still
 * running on another stream is not waited for.  Callers that run the library
 * on several streams and need to attribute a timeout synchronise those
 * streams before calling this, or call it from one thread after all of them.
 */
qk_status qk_get_device_status(qk_stream_t stream);

/*
 * Diagnostic for the failure path: enqueue on `stream` a kernel whose only
 * wait can never complete (an mbarrier nothing arrives on).  Like every wait
 * in the library's kernels it gives up after a wall-clock limit, here
 * `limit_ns` (clamped to 1 us .. 1 s), raises the device status word and
 * returns, so the next qk_get_device_status() reports QK_ERR_TIMEOUT and the
 * CUDA context stays usable.  No fault, trap or unbounded wait is involved.
 * Returns QK_ERR_UNSUPPORTED_DEVICE or QK_ERR_CUDA on launch problems.
 */
qk_status qk_debug_wait_timeout(int64_t limit_ns, qk_stream_t stream);

/*
 * Host-only query (no CUDA call): 1 if an M = 1 problem in format `qtype`
 * (QK_Q4_K / QK_Q6_K; with gateup != 0 the fused gate/up + SwiGLU, Q4_K only)
 * and inner size K runs on the decode GEMV, 0 if it runs on the tensor-core
 * GEMM because the GEMV cannot stage it (the x table of K plus two weight
 * stages must fit in shared memory: K <= 35840 for Q4_K, 35072 for gate/up;
 * Q6_K up to K = 26624 when K / 256 is a multiple of 8, else up to 6912),
 * -1 for an invalid qtype or K.  The answer depends only on these arguments.
 */
int qk_decode_uses_gemv(int qtype, int gateup, int64_t K);

/*
 * Host-only query (no CUDA call), for any M: 1 if an M x N x K problem in
 * format `qtype` (gateup != 0: the fused gate/up + SwiGLU) runs on the
 * CUDA-core-fed GEMV (M <= 8: M = 1 in the decode layout, 2..8 with the
 * tokens in the MMA columns; the x table of M tokens plus two weight stages
 * must fit in shared memory), 0 if it runs on the tensor-core GEMM, -1 for
 * invalid arguments.  qk_decode_uses_gemv(q, g, K) is qk_uses_gemv(q, g, 1, K).
 */
int qk_uses_gemv(int qtype, int gateup, int64_t M, int64_t K);

/*
 * Host-only query: the launch plan the tensor-core GEMM (M > 1, and M = 1
 * problems the GEMV cannot stage) uses for an M x N problem of format
 * `qtype` (gateup != 0: the fused gate/up + SwiGLU, Q4_K only).  Needs no GPU;
 * with one present, the current device's shared-memory limits are used.
 * tcgen05.alloc waits without a time limit until tensor-memory columns are
 * free, so the plan pads a CTA's shared memory until the CTAs that can share
 * an SM fit in its 512 columns together: max_ctas_per_sm * tmem_cols <= 512.
 * Returns QK_ERR_SHAPE for invalid arguments (as qk_matmul_q4k), else QK_OK.
 */
typedef struct qk_gemm_plan_info {
  int token_tile;      /* tokens per CTA tile (the UMMA N dimension), a multiple of 16 */
  int x_stages;        /* activation-tile ring depth */
  int a_stages;        /* dequantized weight-tile ring depth */
  int packed_stages;   /* packed super-block ring depth */
  int a_in_tmem;       /* 1: dequantized weight tiles live in tensor memory, 0: in shared memory */
  int tmem_cols;       /* tensor-memory columns one CTA allocates */
  int smem_bytes;      /* dynamic shared memory per CTA */
  int max_ctas_per_sm; /* CTAs that fit on one SM by shared memory */
} qk_gemm_plan_info;

qk_status qk_gemm_plan(int qtype, int gateup, int64_t M, int64_t N, int64_t K, qk_gemm_plan_info *out);

/* A static, human-readable name for a status code. */
const char *qk_status_string(qk_status status);

/* Library version, major*10000 + minor*100 + patch. */
int qk_version(void);

#ifdef __cplusplus
}
#endif

#endif /* QK_H */
