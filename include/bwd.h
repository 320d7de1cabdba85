/*
 * bwd.h -- C ABI of the GB300 (sm_103a) 8-bit block-wise dynamic Adam library.
 *
 * The method: "8-BIT OPTIMIZERS VIA BLOCK-WISE QUANTIZATION", as summarised on
 * wiki.neutronadmin.com/news/16836.  Adam's two moments (section 一) are kept
 * as 8-bit codes; for the update they are dequantized to fp32, the update
 * runs, and they are quantized again (section 二, opening paragraph).  Codes
 * index a 256-entry dynamic-tree map (section 二 / 动态量化: sign, zero-run
 * exponent, indicator bit, linear fraction; the second moment uses the
 * unsigned variant whose sign bit is one more fraction bit), and every block
 * of 2048 elements carries one fp32 absmax (section 二 / 逐块量化).
 *
 * Conventions shared by every entry point
 *   - Pointers named "device" are CUDA device (or managed) memory of the
 *     CURRENT device; the caller owns them.  The library keeps only its own
 *     immutable code tables (about 26 KB per device, uploaded on first use)
 *     and one fault word (see bwd_check_device).
 *   - Every device operation is enqueued on `stream` (a cudaStream_t; NULL is
 *     the legacy default stream) and returns without waiting for it.  Launch
 *     errors are reported as BWD_ERR_CUDA; faults inside a kernel surface on
 *     the caller's next synchronisation, as for any CUDA work.
 *   - Arguments are checked on the host before anything is enqueued; a
 *     rejected call has no effect.  n == 0 is a successful no-op.
 *   - Every pointer must be aligned to its element size (4 bytes for fp32,
 *     2 for bf16, 8 for int64; BWD_ERR_INVALID_ARG otherwise).  Beyond that
 *     any alignment is accepted: 16-byte aligned pointers (and, per tensor,
 *     full 2048-element blocks) take the vectorised path; other blocks take
 *     an element-wise path with identical results.
 *   - Input and output ranges must not overlap, except where an argument is
 *     documented as updated in place.
 *   - Non-finite inputs are outside the method; they never cause an
 *     out-of-bounds access but their codes are unspecified.
 *   - The first call on a device uploads the tables with a blocking copy, so
 *     it must not happen during CUDA stream capture; bwd_init() does it
 *     explicitly.
 *   - Entry points are thread-safe; bwd_last_error() is per thread.
 */
#ifndef BWD_H
#define BWD_H

#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* Elements per quantization block (section 二 / 逐块量化). */
#define BWD_BLOCK 2048

typedef enum {
  BWD_OK = 0,
  BWD_ERR_INVALID_ARG = 1,       /* null pointer, negative size, bad enum, ... */
  BWD_ERR_UNSUPPORTED_DTYPE = 2, /* gradient dtype not in bwd_dtype          */
  BWD_ERR_CUDA = 3               /* a CUDA runtime call or launch failed      */
} bwd_status;

/* Which dynamic-tree map (section 二 / 动态量化). */
typedef enum {
  BWD_MAP_SIGNED = 0,   /* sign + zero-run exponent + indicator + fraction  */
  BWD_MAP_UNSIGNED = 1  /* the sign bit reused as fraction (second moment)  */
} bwd_map_kind;

/* Element types of gradients and (for bwd_adam8bit_step_multi_ex) of
 * parameters: fp32, bf16, IEEE binary16.  16-bit values widen exactly; 16-bit
 * parameters are rounded back to nearest, ties to even. */
typedef enum { BWD_F32 = 0, BWD_BF16 = 1, BWD_F16 = 2 } bwd_dtype;

/* Adam hyper-parameters (section 一: first and second moment).  `step` is
 * the 1-based index t of the step being taken (bias corrections use it).
 * weight_decay >= 0 is decoupled weight decay (AdamW, an extension of the
 * method): p is first scaled by fp32(1 - lr * weight_decay); 0 gives Adam. */
typedef struct {
  float lr;
  float beta1;
  float beta2;
  float eps;
  float weight_decay;
  int64_t step;
} bwd_adam_hparams;

/* Number of 2048-element blocks of an n-element tensor: ceil(n / 2048).
 * Returns -1 for n < 0. */
int64_t bwd_num_blocks(int64_t n);

/* Host only.  Writes the 256-entry map of `kind` in ascending order (a code
 * is an index into it; the signed map holds -0.0 at 127 and +0.0 at 128) and
 * the 255 decision thresholds, threshold i being the binary32 value nearest
 * to the midpoint of entries i and i+1.  Magnitudes follow the dynamic-tree
 * layout of section 二 / 动态量化 with a decimal zero-run exponent and a
 * linear fraction grid on (0.1, 1] per decade.  Either output may be NULL. */
bwd_status bwd_build_map(bwd_map_kind kind, float* map_out /*[256]*/,
                         float* thresholds_out /*[255]*/);

/* Uploads the code tables to the current device if not done yet (blocking).
 * Optional: every entry point below does it on first use. */
bwd_status bwd_init(void);

/* Block-wise quantization (section 二 / 逐块量化 and 动态量化).
 *   x      : device, float[n], read only.
 *   codes  : device, uint8[n], written: index of the nearest map entry to
 *            x / absmax (binary32 IEEE division; a value exactly on a
 *            threshold takes the higher code; +-0 take the code of +0).
 *   absmax : device, float[ceil(n/2048)], written: max |x| of each block
 *            (the last block may be partial).  A block whose absmax is 0
 *            gets the code of +0.0 everywhere. */
bwd_status bwd_quantize_blockwise(const float* x, int64_t n, bwd_map_kind kind,
                                  uint8_t* codes, float* absmax, void* stream);

/* Block-wise dequantization (section 一: back from codes to values).
 *   codes  : device, uint8[n]; absmax: device, float[ceil(n/2048)].
 *   y      : device, float[n], written: map[code] * absmax[block] (one
 *            binary32 multiply). */
bwd_status bwd_dequantize_blockwise(const uint8_t* codes, const float* absmax,
                                    int64_t n, bwd_map_kind kind, float* y,
                                    void* stream);

/* State before the first step: m codes := code of +0.0 in the signed map,
 * v codes := code of 0 in the unsigned map, both absmax := 0.
 *   m_codes, v_codes : device uint8[n];  m_absmax, v_absmax : device
 *   float[ceil(n/2048)].  All written. */
bwd_status bwd_state_init(uint8_t* m_codes, float* m_absmax, uint8_t* v_codes,
                          float* v_absmax, int64_t n, void* stream);

/* One 8-bit Adam step on one flat tensor (section 二, opening paragraph):
 * dequantize m (signed map) and v (unsigned map), run Adam in fp32,
 *     m = b1 m + (1-b1) g;  v = b2 v + ((1-b2) g) g;
 *     p = p d - (s m) / (sqrt(v) / c + eps),
 * with s = fp32(lr / (1 - b1^t)), c = fp32(sqrt(1 - b2^t)) and the decay
 * factor d = fp32(1 - lr wd) formed in binary64 on the host; then requantize
 * m and v block by block with fresh absmax.  m and v take one binary32
 * rounding per operation in that order, so the new codes and absmax are
 * exactly those of IEEE arithmetic; the parameter update uses approximate
 * (sqrt / rcp) arithmetic and is within a few ulps of the update term.
 *   p                : device float[n], updated in place.
 *   g                : device, float[n], bf16[n] or fp16[n] per g_dtype, read
 *                      only.
 *   m_codes, v_codes : device uint8[n], updated in place.
 *   m_absmax,v_absmax: device float[ceil(n/2048)], updated in place.
 *   hp               : host pointer; hp->step >= 1, lr and eps finite,
 *                      eps >= 0, betas in [0, 1), weight_decay finite >= 0. */
bwd_status bwd_adam8bit_step(float* p, const void* g, bwd_dtype g_dtype,
                             uint8_t* m_codes, float* m_absmax,
                             uint8_t* v_codes, float* v_absmax, int64_t n,
                             const bwd_adam_hparams* hp, void* stream);

/* The same step over a list of tensors in as few launches as the kernel
 * parameter space allows (448 tensors per launch).  Blocks never span two
 * tensors.  All arrays are HOST arrays of length num_tensors holding device
 * pointers (or sizes); each tensor follows the single-tensor contract above.
 * Tensors with n == 0 are skipped; num_tensors == 0 is a no-op. */
bwd_status bwd_adam8bit_step_multi(int32_t num_tensors, float* const* p,
                                   const void* const* g, bwd_dtype g_dtype,
                                   uint8_t* const* m_codes,
                                   float* const* m_absmax,
                                   uint8_t* const* v_codes,
                                   float* const* v_absmax, const int64_t* n,
                                   const bwd_adam_hparams* hp, void* stream);

/* The multi-tensor step with the parameter type given: p_dtype BWD_F32
 * (as bwd_adam8bit_step_multi), BWD_BF16 or BWD_F16.  16-bit parameters are
 * widened to fp32 for the update and stored back rounded to nearest even
 * (the page's low-precision state with a high-precision update, section 二,
 * opening paragraph, which names FP16); codes and absmax are the same as
 * with fp32 parameters.
 *   p : HOST array of num_tensors device pointers to fp32[n], bf16[n] or
 *       fp16[n] parameters, updated in place.  Other arguments as above. */
bwd_status bwd_adam8bit_step_multi_ex(int32_t num_tensors, void* const* p,
                                      bwd_dtype p_dtype, const void* const* g,
                                      bwd_dtype g_dtype, uint8_t* const* m_codes,
                                      float* const* m_absmax,
                                      uint8_t* const* v_codes,
                                      float* const* v_absmax, const int64_t* n,
                                      const bwd_adam_hparams* hp, void* stream);

/* The same with every gradient multiplied by s = *grad_scale first (one
 * binary32 product), a factor in device memory such as bwd_grad_norm's.
 *   grad_scale : device float[1], read by the kernel, or NULL for
 *                bwd_adam8bit_step_multi_ex.  Where it is infinite or NaN the
 *                call writes nothing. */
bwd_status bwd_adam8bit_step_multi_scaled(
    int32_t num_tensors, void* const* p, bwd_dtype p_dtype,
    const void* const* g, bwd_dtype g_dtype, uint8_t* const* m_codes,
    float* const* m_absmax, uint8_t* const* v_codes, float* const* v_absmax,
    const int64_t* n, const float* grad_scale, const bwd_adam_hparams* hp,
    void* stream);

/* The same with the number of steps taken held in device memory, because where
 * *grad_scale is not finite nothing is written and the step is not counted,
 * which the host does not know; and so that a captured call can be replayed
 * as the next step.
 *   grad_scale : as above; NULL for 1.
 *   count      : device, 16 bytes, 8-byte aligned: an int64_t, the steps taken
 *                so far, and eight bytes that the call writes.  The call takes
 *                step *count + 1 and leaves *count that, or as it was.
 *                hp->step is not read. */
bwd_status bwd_adam8bit_step_multi_counted(
    int32_t num_tensors, void* const* p, bwd_dtype p_dtype,
    const void* const* g, bwd_dtype g_dtype, uint8_t* const* m_codes,
    float* const* m_absmax, uint8_t* const* v_codes, float* const* v_absmax,
    const int64_t* n, const float* grad_scale, void* count,
    const bwd_adam_hparams* hp, void* stream);

/* ------------------------------------------------------------------------
 * ZeRO-style sharding of the step over P processes ("Яндекс Публикует ЯЛМ
 * 100Б", section "ZeRO" under "Случай с несколькими графическими
 * процессорами": each process keeps the values and optimizer state of its own
 * group of parameters and alone updates them, so its step is O(N / P); the
 * gradients are reduced before the step and the parameters gathered after
 * it).  Blocks are independent (section 二 / 逐块量化 of the 8-bit optimizer
 * page), so the split follows block boundaries and a rank's step over its
 * pieces (bwd_adam8bit_step_multi / _ex, pointers offset by `offset`
 * elements) equals the unsharded step on those elements bit for bit.
 *
 * Layout: in a padded flat space tensor i occupies the blocks
 * [B_i, B_i + ceil(n_i / 2048)), B the prefix sums of the block counts and NB
 * their total; rank r owns the K = ceil(NB / world) blocks [r K, (r + 1) K)
 * clipped to NB (the last ranks may own fewer, or none), so padded buffers of
 * world * K * 2048 elements split into equal per-rank slices.
 *   n               : HOST int64[num_tensors], tensor sizes (0 allowed).
 *   world, rank     : 1 <= world, 0 <= rank < world.
 *   blocks_per_rank : HOST int64 out, K (may be NULL).
 *   num_pieces      : HOST int32 out, the tensors the rank's blocks touch.
 *   tensor, offset, count : HOST arrays of capacity num_tensors, written
 *            (each may be NULL): piece j is the elements
 *            [offset[j], offset[j] + count[j]) of tensor tensor[j]; offsets
 *            are multiples of 2048; pieces ascend in tensor order.
 * Host only (no device is touched).  BWD_ERR_INVALID_ARG for a negative size,
 * a NULL pointer, world < 1, rank outside [0, world) or a total that
 * overflows. */
bwd_status bwd_zero_shard(int32_t num_tensors, const int64_t* n, int32_t world,
                          int32_t rank, int64_t* blocks_per_rank,
                          int32_t* num_pieces, int32_t* tensor,
                          int64_t* offset, int64_t* count);

/* ------------------------------------------------------------------------
 * Stable embedding layer (section 二 / 稳定的词嵌入层): the embedding weight
 * is initialised Xavier-uniform and a layer normalisation follows the
 * lookup, so that the layer's output has variance close to 1.
 *   weight : device fp32[V * D], row-major (row v = embedding of token v).
 *   gamma, beta : device fp32[D], the normalisation's scale and shift.
 *   ids    : device int64[T] token ids.  An id outside [0, V) is outside
 *            the method: its output row is NaN (no access leaves the
 *            weight) and the backward pass skips it.
 * D a multiple of 4 and at most 4096 with 16-byte aligned weight, gamma,
 * beta / dy, y / dweight takes the vectorised path; any other shape takes an
 * element-wise path with the same arithmetic.  All fp32, eps as given.
 * Errors: BWD_ERR_INVALID_ARG for V < 1, D < 1, T < 0, V * D or T * D
 * overflowing int64, a NULL pointer, a non-finite or negative eps. */

/* Xavier-uniform initialisation from caller-supplied random words:
 * weight[i] = fp32((2 u_i - 1) * b), u_i = (words[i] >> 8) * 2^-24 and
 * b = fp32(sqrt(6 / (V + D))) (Glorot's bound for fan-in D and fan-out V;
 * 2 u - 1 is exact, so each weight takes one rounding).
 *   words  : device uint32[V * D], e.g. from any uniform 32-bit generator.
 *   weight : device fp32[V * D], written. */
bwd_status bwd_embedding_init(const uint32_t* words, int64_t num_embeddings,
                              int64_t dim, float* weight, void* stream);

/* Host only: the bound b above, or -1 for V < 1 or D < 1. */
float bwd_embedding_xavier_bound(int64_t num_embeddings, int64_t dim);

/* Forward: for each token t with x = weight[ids[t]],
 *   mean = sum(x) / D,  var = sum((x - mean)^2) / D,
 *   rstd = 1 / sqrt(var + eps),  y = (x - mean) * rstd * gamma + beta.
 *   y    : device fp32[T * D], written.
 *   mean, rstd : device fp32[T], written (the backward pass reads them);
 *          either may be NULL when no backward pass follows.
 * Row statistics are reduced in a fixed order: results are deterministic. */
bwd_status bwd_embedding_forward(const int64_t* ids, int64_t num_tokens,
                                 const float* weight, int64_t num_embeddings,
                                 int64_t dim, const float* gamma,
                                 const float* beta, float eps, float* y,
                                 float* mean, float* rstd, void* stream);

/* Backward: with xhat = (x - mean) * rstd (mean, rstd from the forward call)
 * and g = dy * gamma, per token
 *   dx = rstd * (g - mean(g) - xhat * mean(g * xhat)),
 * ACCUMULATED into the caller's buffers (zero them for a fresh gradient):
 *   dweight[ids[t]] += dx   (device fp32[V * D]; repeated ids add up),
 *   dgamma += sum_t dy * xhat,  dbeta += sum_t dy   (device fp32[D]).
 *   dy : device fp32[T * D].
 * The adds are atomic, so their order, and the last bits of dweight, dgamma
 * and dbeta, may differ between runs. */
bwd_status bwd_embedding_backward(const int64_t* ids, int64_t num_tokens,
                                  const float* weight, int64_t num_embeddings,
                                  int64_t dim, const float* gamma,
                                  const float* mean, const float* rstd,
                                  const float* dy, float* dweight,
                                  float* dgamma, float* dbeta, void* stream);

/* Hyper-parameters of the step below: bwd_adam_hparams with its numbers in
 * binary64, so that 1 - beta and the bias corrections are those of the beta
 * meant (a binary32 0.999 is off by 1.3e-8, its 1 - beta by 1.3e-5 of it). */
typedef struct {
  double lr;
  double beta1;
  double beta2;
  double eps;
  double weight_decay;
  int64_t step;
} bwd_adamw_hparams;

/* ------------------------------------------------------------------------
 * AdamW with both moments in fp32, for the tensors of a run whose moments
 * stay in 32 bits (an embedding, norms, biases), and the gradients' norm.
 *
 * One step over a list of tensors (480 per launch), in place:
 *     g' = s g;  m = b1 m + (1-b1) g';  v = b2 v + ((1-b2) g') g';
 *     p = p d - step m / (sqrt(v) / c + eps)
 * with step, c and d formed in binary64 on the host as for
 * bwd_adam8bit_step (each scalar rounded once) and s = *grad_scale.  m and v
 * take one binary32 rounding per operation in that order.  Arrays are HOST arrays
 * of length num_tensors.
 *   p          : device pointers to n[i] values of p_dtype, updated in place
 *                (16-bit ones are widened and rounded back to nearest even).
 *   g          : device pointers to n[i] values of g_dtype, read only.
 *   m, v       : device pointers to float[n[i]], updated in place.
 *   grad_scale : device float[1], read by the kernel, or NULL for 1.  Where
 *                it is infinite or NaN the call writes nothing.
 * A NaN or infinite gradient makes its own element's state and parameter
 * NaN or infinite and no other. */
bwd_status bwd_adam32_step_multi(int32_t num_tensors, void* const* p,
                                 bwd_dtype p_dtype, const void* const* g,
                                 bwd_dtype g_dtype, float* const* m,
                                 float* const* v, const int64_t* n,
                                 const float* grad_scale,
                                 const bwd_adamw_hparams* hp, void* stream);

/* The same with the number of steps taken in device memory, as for
 * bwd_adam8bit_step_multi_counted. */
bwd_status bwd_adam32_step_multi_counted(
    int32_t num_tensors, void* const* p, bwd_dtype p_dtype,
    const void* const* g, bwd_dtype g_dtype, float* const* m, float* const* v,
    const int64_t* n, const float* grad_scale, void* count,
    const bwd_adamw_hparams* hp, void* stream);

/* Bytes of the workspace of bwd_grad_norm (-1 for num_tensors < 0). */
int64_t bwd_grad_norm_work_bytes(int32_t num_tensors);

/* 2-norm of all elements of a list of gradients, and the factor that brings
 * it to max_norm at most:
 *     norm = sqrt(sum (g / loss_scale)^2),
 *     factor = min(1, max_norm / (norm + 1e-6)) / loss_scale,
 * NaN where the norm is not finite, so that a step that reads it as its
 * grad_scale writes nothing.  Sums are fp32 within 64 bytes of a thread, or
 * binary64 where those squares leave fp32's range, and binary64 above, in a
 * fixed order: results are deterministic, and elements of any finite
 * magnitude count.
 *   g_dtype : HOST array, the bwd_dtype of each tensor.
 *   factor, norm : device float[1] each, written.
 *   work : device, 16-byte aligned, bwd_grad_norm_work_bytes(num_tensors)
 *          bytes, whose first 16 are zero before the first call; each call
 *          leaves them zero.  Calls that may run at the same time need one
 *          each.
 *   max_norm > 0 (infinity: no clipping), loss_scale > 0 and finite, as is
 *   1 / loss_scale.  num_tensors == 0 gives norm 0. */
bwd_status bwd_grad_norm(int32_t num_tensors, const void* const* g,
                         const int32_t* g_dtype, const int64_t* n, float max_norm,
                         float loss_scale, float* factor, float* norm,
                         void* work, void* stream);

/* ------------------------------------------------------------------------
 * 8-bit floating point (e4m3) with a power-of-two scale for each block of
 * 128: section 二 / 逐块量化's block-wise scaling applied to the operands of a
 * linear layer's products.
 *
 * A block's scale is 2^e, e the smallest integer >= -127 for which no
 * magnitude in the block exceeds 448 * 2^e; a value's code is the e4m3 number
 * nearest to x * 2^-e, ties to even.  A block with an infinity or a NaN has
 * the NaN scale (byte 255) and NaN codes: every product with it is NaN.
 *
 * Code array of a rows x cols matrix: uint8[rows][pitch], 16-byte aligned,
 * pitch = bwd_fp8_pitch(cols): cols rounded up to 128, or to 16 for up to 64
 * of them.  A product reads whole rows: the bytes past cols are zero (NaN
 * codes beside NaN codes will do), as bwd_fp8_quantize writes them.
 *
 * Scale array for `count` lines of `length` elements, each line in blocks of
 * 128: bwd_fp8_scale_bytes(count, length) bytes, 16-byte aligned; the byte
 * e + 127 of line r, block k is at
 *     ((r / 128) * G + k / 4) * 512 + (r % 32) * 16 + (r / 32 % 4) * 4 + k % 4
 * with G = ceil(ceil(length / 128) / 4), the order in which the matrix
 * instruction's scale memory is filled. */
#define BWD_FP8_ROWS 1  /* blocks of 1 x 128: lines are the rows           */
#define BWD_FP8_COLS 2  /* blocks of 128 x 1: lines are the columns        */
#define BWD_FP8_TILES 4 /* blocks of 128 x 128, with scales for both lines */

/* Both -1 for a negative size or one above 2^30. */
int64_t bwd_fp8_pitch(int64_t cols);
int64_t bwd_fp8_scale_bytes(int64_t count, int64_t length);

/* Quantizes x (device, rows x cols, `ld` elements between rows).
 *   blocks : BWD_FP8_ROWS, BWD_FP8_COLS, both of them together, or
 *            BWD_FP8_TILES.
 *   row_codes, row_scales : written for BWD_FP8_ROWS and BWD_FP8_TILES;
 *            scales of `rows` lines of `cols` elements.
 *   col_codes : written for BWD_FP8_COLS.
 *   col_scales: written for BWD_FP8_COLS and BWD_FP8_TILES; scales of `cols`
 *            lines of `rows` elements.
 *   col_sums : with BWD_FP8_COLS, or NULL: cols values of x's type, written:
 *            the columns' sums (summed in fp32; a bias's gradient).
 *   col_sums_work : device float[ceil(rows / 128) * cols] if col_sums is
 *            given.
 * At most 65535 * 128 rows. */
bwd_status bwd_fp8_quantize(const void* x, bwd_dtype dtype, int64_t rows,
                            int64_t cols, int64_t ld, int32_t blocks,
                            uint8_t* row_codes, uint8_t* row_scales,
                            uint8_t* col_codes, uint8_t* col_scales,
                            void* col_sums, float* col_sums_work,
                            void* stream);

/* code * 2^e as out[rows][cols] (contiguous) of the given type, rounded to
 * nearest once; along_rows says which lines the scales belong to (1: rows). */
bwd_status bwd_fp8_dequantize(const uint8_t* codes, const uint8_t* scales,
                              int32_t along_rows, int64_t rows, int64_t cols,
                              void* out, bwd_dtype dtype, void* stream);

/* out[i, j] = sum_l A(i, l) B(j, l) + bias[j], i < m, j < n, l < k.
 *   a, a_scales : codes and scales of m lines of k elements.  a_trans 0: the
 *            lines are the rows of an m x k matrix; 1: they are the columns
 *            of a k x m matrix.  b the same with n for m.
 *   bias : device, n values of the output's type, or NULL.
 *   out  : device, m x n values of `dtype`, `ldo` elements between rows.
 * Products are exact, sums are held in fp32, and the result is rounded once;
 * the order of the sums is fixed.  The matrix instruction truncates its fp32
 * additions and so loses some 1.9e-10 of a sum of like signs for each product
 * (measured: 7.6e-7 after 4,096, 2.0e-5 after 65,536): fp32 results leave it
 * every 2,048 products and are then added up to nearest; 16-bit results, whose
 * own rounding is 4.9e-4 or more, may take all of a sum in it. */
bwd_status bwd_fp8_matmul(int64_t m, int64_t n, int64_t k, const uint8_t* a,
                          int32_t a_trans, const uint8_t* a_scales,
                          const uint8_t* b, int32_t b_trans,
                          const uint8_t* b_scales, const void* bias, void* out,
                          int64_t ldo, bwd_dtype dtype, void* stream);

/* A linear layer's forward pass in one call: y = Q(x) W^T + bias, x
 * (rows x cols) quantized in blocks of 1 x 128 in the workspace.
 *   w, w_scales : codes and scales of n lines of cols elements (BWD_FP8_ROWS
 *            or BWD_FP8_TILES of an n x cols weight).
 *   bias : n values of x's type, or NULL.   y : rows x n of x's type.
 *   x_col_codes, x_col_scales : both NULL, or written as for BWD_FP8_COLS
 *            (the backward pass reads them).
 *   work : device, 16-byte aligned, bwd_fp8_linear_work_bytes(rows, cols)
 *            bytes; none, and NULL will do, for up to 16 rows of up to
 *            245,760 elements, which the product's kernel quantizes itself. */
int64_t bwd_fp8_linear_work_bytes(int64_t rows, int64_t cols);
bwd_status bwd_fp8_linear(const void* x, bwd_dtype dtype, int64_t rows,
                          int64_t cols, int64_t ld, const uint8_t* w,
                          const uint8_t* w_scales, int64_t n, const void* bias,
                          void* y, int64_t ldy, uint8_t* x_col_codes,
                          uint8_t* x_col_scales, void* work, void* stream);

/* Its backward pass: dy (rows x n) is quantized once in both forms, then
 *     dx = Q(dy) W           rows x k, `lddx` between rows, or NULL
 *     dw = Q(dy)^T Q(x)      n x k, `lddw` between rows, or NULL
 *     dbias = sum of dy's rows   n values, or NULL
 * all of dy's type.
 *   w, w_col_scales : codes and scales of the k columns of the n x k weight
 *            (BWD_FP8_TILES or BWD_FP8_COLS); read for dx.
 *   x_col_codes, x_col_scales : of x's k columns; read for dw.
 *   work : device, 16-byte aligned,
 *            bwd_fp8_linear_backward_work_bytes(rows, n). */
int64_t bwd_fp8_linear_backward_work_bytes(int64_t rows, int64_t n);
bwd_status bwd_fp8_linear_backward(const void* dy, bwd_dtype dtype,
                                   int64_t rows, int64_t n, int64_t ld,
                                   const uint8_t* w,
                                   const uint8_t* w_col_scales,
                                   const uint8_t* x_col_codes,
                                   const uint8_t* x_col_scales, int64_t k,
                                   void* dx, int64_t lddx, void* dw,
                                   int64_t lddw, void* dbias, void* work,
                                   void* stream);

/* ------------------------------------------------------------------------
 * Microscaled 4-bit floating point.  A block of 1 x 32 elements of a row has
 * the scale 2^e, e >= -127 the smallest for which no magnitude of the block
 * exceeds 6 * 2^e, and each element the e2m1 code (0, 0.5, 1, 1.5, 2, 3, 4, 6
 * and their negatives) nearest to x 2^-e, ties to the even code.  A block with
 * an infinity or a NaN stands for NaN throughout.
 *   codes  : two to a byte, the earlier column in the low half; rows start
 *            bwd_fp4_pitch(cols) bytes apart (16-byte aligned), the rest of a
 *            row's bytes are zero.
 *   scales : e + 127 of row r's block k (columns 32 k and on) at byte
 *            ((r / 128) G + k / 4) 512 + (r % 32) 16 + (r / 32 % 4) 4 + k % 4,
 *            G = 2 ceil(cols / 256); bwd_fp4_scale_bytes(rows, cols) in all.
 *            Of existing rows, blocks past the last column have the byte 0;
 *            the bytes of rows that do not exist are not written. */
int64_t bwd_fp4_pitch(int64_t cols);
int64_t bwd_fp4_scale_bytes(int64_t rows, int64_t cols);

/* x: device, rows x cols values of `dtype`, `ld` elements between rows; at most
 * 65535 * 32 = 2,097,120 rows here, to read back and for bwd_fp4_linear. */
bwd_status bwd_fp4_quantize(const void* x, bwd_dtype dtype, int64_t rows,
                            int64_t cols, int64_t ld, uint8_t* codes,
                            uint8_t* scales, void* stream);

/* out: device, rows x cols values of `dtype`, contiguous. */
bwd_status bwd_fp4_dequantize(const uint8_t* codes, const uint8_t* scales,
                              int64_t rows, int64_t cols, void* out,
                              bwd_dtype dtype, void* stream);

/* out[i, j] = sum_l A(i, l) B(j, l) + bias[j], i < m, j < n, l < k, for
 * quantized A (m x k) and B (n x k).
 *   bias : device, n values of `dtype`, or NULL.
 *   out  : device, m x n values of `dtype`, `ldo` elements between rows.
 * Products are exact, sums are held in fp32 (the matrix instruction truncates
 * its additions; fp32 results leave it every 2,048 products and are then added
 * up to nearest), and the result is rounded once; the order is fixed. */
bwd_status bwd_fp4_matmul(int64_t m, int64_t n, int64_t k, const uint8_t* a,
                          const uint8_t* a_scales, const uint8_t* b,
                          const uint8_t* b_scales, const void* bias, void* out,
                          int64_t ldo, bwd_dtype dtype, void* stream);

/* y = Q(x) W^T + bias in one call, x (rows x cols) quantized in the workspace.
 *   w, w_scales : of the n x cols weight.   y : rows x n of x's type.
 *   work : device, 16-byte aligned, bwd_fp4_linear_work_bytes(rows, cols)
 *          bytes; none, and NULL will do, for up to 8 rows of up to 229,376
 *          elements, which the product's kernel quantizes itself. */
int64_t bwd_fp4_linear_work_bytes(int64_t rows, int64_t cols);
bwd_status bwd_fp4_linear(const void* x, bwd_dtype dtype, int64_t rows,
                          int64_t cols, int64_t ld, const uint8_t* w,
                          const uint8_t* w_scales, int64_t n, const void* bias,
                          void* y, int64_t ldy, void* work, void* stream);

/* ------------------------------------------------------------------------
 * Layer normalisation over the rows of a matrix:
 *     mean = sum x / D;  var = sum (x - mean)^2 / D;  rstd = (var + eps)^-1/2
 *     xh = (x - mean) rstd;  y = xh gamma + beta
 *   x    : device, rows x width values of `dtype`, `ldx` elements between
 *          rows; width at most 16384.
 *   gamma, beta : device, width values of `vector_dtype`, which is BWD_F32 or
 *          x's; NULL for 1 and 0.
 *   y    : device, rows x width values of `dtype`, written.
 *   mean, rstd : device float[rows], written, or NULL.
 * Statistics are held in fp32, the variance is of the centred values. */
bwd_status bwd_norm_forward(const void* x, bwd_dtype dtype, int64_t rows,
                            int64_t width, int64_t ldx, const void* gamma,
                            const void* beta, bwd_dtype vector_dtype, float eps,
                            void* y, float* mean, float* rstd, void* stream);

/* Its gradients for the given statistics:
 *     h = dy gamma
 *     dx = rstd (h - sum h / D - xh sum(h xh) / D)   rows x width, or NULL
 *     dgamma = sum over rows of dy xh    width values of `vector_dtype`, or NULL
 *     dbeta = sum over rows of dy        the same
 * all written, in a fixed order of sums.
 *   work : device, 4-byte aligned, bwd_norm_backward_work_bytes(rows, width);
 *          read and written where dgamma or dbeta is. */
int64_t bwd_norm_backward_work_bytes(int64_t rows, int64_t width);
bwd_status bwd_norm_backward(const void* dy, const void* x, bwd_dtype dtype,
                             int64_t rows, int64_t width, int64_t lddy,
                             int64_t ldx, const void* gamma,
                             bwd_dtype vector_dtype, const float* mean,
                             const float* rstd, void* dx, void* dgamma,
                             void* dbeta, void* work, void* stream);

/* ------------------------------------------------------------------------
 * Orthogonalised updates.  For each matrix G (rows x cols, contiguous):
 *     X = G / (|G| + 1e-7)   Frobenius norm; G^T where rows > cols
 *     `steps` times:  A = X X^T;  X = a X + (b A + c A A) X
 * with (a, b, c) = (3.4445, -4.7750, 2.0315), and the result X (or X^T).
 * Five steps bring singular values above 1e-3 of the norm to 0.7 ... 1.2.
 *   g, out : HOST arrays of device pointers to rows[i] x cols[i] values of
 *            `dtype`; out[i] may be g[i].  Matrices of one shape, or of its
 *            transpose, are worked on together, up to 64 of them.
 *   rows, cols : HOST arrays, at most 65536 each; an empty matrix is left out.
 *   work : device, 256-byte aligned, bwd_orthogonalize_work_bytes(...) bytes
 *          (-1 for a bad argument); calls that share it are ordered by the
 *          caller.  A matrix of m x n, m <= n, takes 8 m (n + m) bytes, with
 *          n and m in the sums rounded up to 64, and 8 m m more where 2 m <= n
 *          <= 16 m; up to 64 matrices are worked on together, of those that
 *          are not small as many as 4 GB hold.
 * Products are of pairs of fp16 values (22 bits), added in fp32 by the matrix
 * instruction, which truncates; sums leave it every 128 products and are then
 * added up to nearest.  A result is off by 1e-6 to 8e-6 of its norm before it
 * is rounded, as in fp32, a bf16 one with 2 <= n / m <= 16 by up to 1e-4.  A matrix with a
 * NaN or an infinity comes out NaN, the others are not touched by it. */
int64_t bwd_orthogonalize_work_bytes(int32_t count, const int64_t* rows,
                                     const int64_t* cols);
bwd_status bwd_orthogonalize(int32_t count, const void* const* g,
                             bwd_dtype dtype, const int64_t* rows,
                             const int64_t* cols, int32_t steps,
                             void* const* out, void* work, void* stream);

/* Hyper-parameters of the step below.  `rms` is the root mean square that an
 * update of full rank is scaled to, before lr (0.2: that of AdamW's). */
typedef struct {
  double lr;
  double momentum;
  double weight_decay;
  double rms;
  int32_t nesterov;
  int32_t steps;
  int64_t work_most; /* bytes that matrices worked on together may take of
                        work, a single one aside; 0 for 4 GB */
} bwd_muon_hparams;

/* One step over a list of matrices, in place:
 *     m = mu m + s g;   u = s g + mu m (nesterov), or m
 *     p = p (1 - lr weight_decay) - lr rms sqrt(max(rows, cols)) O(u)
 * with O as above, formed to the precision that p_dtype asks for.
 *   p, g, m : HOST arrays of device pointers to rows[i] x cols[i] contiguous
 *             values of p_dtype, g_dtype and float; p and m are updated.
 *   grad_scale : device float[1], s, read by the kernels, or NULL for 1.
 *             Where it is infinite or NaN the call writes nothing but work.
 *   work : as for bwd_orthogonalize, bwd_muon_work_bytes(...) bytes for the
 *          hyper-parameters' work_most. */
int64_t bwd_muon_work_bytes(int32_t count, const int64_t* rows,
                            const int64_t* cols, int64_t work_most);
bwd_status bwd_muon_step(int32_t count, void* const* p, bwd_dtype p_dtype,
                         const void* const* g, bwd_dtype g_dtype,
                         float* const* m, const int64_t* rows,
                         const int64_t* cols, const float* grad_scale,
                         const bwd_muon_hparams* hp, void* work, void* stream);

/* Waits for `stream` and reports whether a bounded wait inside one of the
 * library's kernels gave up since the last check (the staged embedding
 * backward and the matrix products wait for their own copies and products; each
 * wait gives up after about a second, flags the device and lets the kernel
 * return).  BWD_OK, or
 * BWD_ERR_CUDA with bwd_last_error() describing it; the flag is cleared.
 * Blocking; not callable during stream capture. */
bwd_status bwd_check_device(void* stream);

/* Self-test of the bounded waits: enqueues one kernel that waits for an
 * mbarrier phase nothing completes.  Its wait gives up after about a second,
 * sets the fault word and returns (no trap, the context stays usable); the
 * next bwd_check_device therefore returns BWD_ERR_CUDA and clears the word.
 * For tests and diagnostics; no counterpart in the method. */
bwd_status bwd_selftest_bounded_wait(void* stream);

/* Static description of a status code. */
const char* bwd_status_string(bwd_status status);

/* Detail of the last failed call on this thread ("" if none). */
const char* bwd_last_error(void);

#ifdef __cplusplus
}
#endif

#endif /* BWD_H */
