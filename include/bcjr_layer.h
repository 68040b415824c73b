/*
 * bcjr_layer.h -- C ABI of the calls around a quantised layer: the optimiser
 * step that trains its weight preimages and codebook, the 4-bit group
 * quantiser and the packing of hard-decoded trellis states, and the products
 * of a few tokens with either kind of packed weights.
 *
 * The conventions are those of bcjr.h: device pointers to row-major
 * contiguous buffers of the caller on the current device, asynchronous on
 * `stream`, argument errors found on the host before anything is launched,
 * nothing allocated, nothing kept.  None of these calls needs a workspace,
 * and all of them may be captured into a CUDA graph.
 */
#ifndef BCJR_LAYER_H
#define BCJR_LAYER_H

#include "bcjr.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef enum { BCJR_F32 = 0, BCJR_F16 = 1, BCJR_BF16 = 2 } bcjr_dtype;

/* One tensor of an optimiser step. */
typedef struct {
  void* param;       /* [numel] of the call's parameter type, updated in place */
  const void* grad;  /* [numel] of the call's gradient type; NULL: this tensor is left as it is */
  int64_t numel;     /* >= 0 */
} bcjr_adamw_tensor;

typedef struct {
  double lr, beta1, beta2, eps, weight_decay;
  int64_t step;             /* 1 for the first step; ignored when step_ptr is given */
  const int64_t* step_ptr;  /* device, or NULL: the step count, read when the kernel runs (for captured graphs) */
  const float* grad_scale;  /* device, or NULL: every gradient is multiplied by *grad_scale */
  uint32_t seed;            /* of the stochastic rounding of 8-bit states */
} bcjr_adamw_options;

/*
 * One AdamW step of n_tensors tensors (`tensors` is a HOST array):
 *   g' = g * grad_scale,  m = b1 m + (1 - b1) g',  v = b2 v + (1 - b2) g'^2,
 *   p = p (1 - lr wd) - lr / (1 - b1^t) * m / (sqrt(v) / sqrt(1 - b2^t) + eps),
 * computed in float32 and p rounded once to its type.  An eps between 0 and
 * 2^-126 counts as 2^-126; with eps 0 an element whose v is 0 becomes a NaN, as
 * 0 / 0 does.
 *
 * The states of all tensors lie in one flat array each, tensor i starting at
 * element 256 * sum_{j < i} ceil(numel_j / 256); what lies between a tensor's
 * end and the next one's start is padding (zeros on entry; stays zero).
 *   state_bits 32: first = m, second = v, float32; scales = NULL.
 *   state_bits 8:  first, second = e4m3 codes (one byte each) of m and of
 *     r = sqrt(v), scales = float32 [2][blocks]: m = code * scales[0][b],
 *     r = code * scales[1][b] for the elements of block b (256 elements).
 *     A block's scale is its largest |m| (r) / 448; a block whose largest is
 *     under 2^-100 holds zeros.  Codes are rounded stochastically, with 16
 *     bits of a hash of (seed, step, flat element index), so the expected
 *     value of a code is the number it stands for and averages over many
 *     steps keep moving when a step's change is smaller than a code; r > 0
 *     never becomes 0, so that no later update divides by eps alone.
 *     Where v overflows (gradients beyond 2^64), the step of that element is 0 as
 *     with 32 bits; its block's scale of r becomes a NaN, and the block's
 *     parameters with it in the next step.  A gradient that is not finite makes
 *     its own parameter NaN and both scales of its block not finite.
 * Types: param and grad float32; param f32 with 16-bit grads; 16-bit param
 * with grads of the same type or float32.  Parameters need only the alignment of their
 * type; the states 16 bytes.  Parameters must not overlap one another, nor the
 * states one another, a parameter or a gradient.
 */
bcjr_status bcjr_adamw_step(const bcjr_adamw_tensor* tensors, int n_tensors, int param_dtype,
                            int grad_dtype, int state_bits, void* first, void* second,
                            float* scales, const bcjr_adamw_options* opt, bcjr_stream_t stream);

/*
 * 4-bit weights in groups along a row.  A group is group_size columns: 32, 64,
 * a multiple of 128, or 0 for the whole row; the last group of a row may be
 * shorter.  scales [groups][rows] (f32, f16 or bf16); zeros [groups][rows]
 * uint8 in 0..15, or NULL for 8 everywhere:
 *   w[r][c] = (q[r][c] - zeros[g][r]) * scales[g][r],  q in 0..15, g = c / group_size.
 *
 * packed [ceil(rows/16)][ceil(cols/128)][1024] bytes: the tile of 16 rows and
 * 128 columns as the tensor-core fragments read it.  Byte
 *   512 h + 64 i + 16 t + 4 j + b   (h < 2, i < 8, t < 4, j < 4, b < 4)
 * holds two codes of row 8 h + i, columns 32 j + 8 t + o: the one at nibble
 * e = 2 b (low) and e = 2 b + 1 (high) of the 32-bit word, with o = 2 e for
 * e < 4 and o = 2 (e - 4) + 1 else.  Codes outside the matrix are 8.
 */

/*
 * Round-to-nearest quantisation of w [rows][cols] into that form.
 *   zeros == NULL: scale = max |w| / 7, q = rint(w / scale) + 8;
 *   else lo = min(w, 0), hi = max(w, 0): scale = (hi - lo) / 15,
 *   zero = rint(-lo / scale), q = rint(w / scale) + zero; q clamped to 0..15.
 * All in float32: the scale is the product with the float32 next to 1/7 (1/15),
 * rounded to its type before the codes are taken, and a code is rint(w * (1 /
 * scale)), which differs from the quotient's only next to a tie.  Where the scale is 0
 * the codes are the zero point.  A group that holds a NaN or an infinity gets
 * a scale that is not finite, and so does one whose range or scale overflows
 * float32 or the scale's type.
 */
bcjr_status bcjr_int4_quantize(const void* w, int w_dtype, int rows, int cols, int group_size,
                               void* packed, void* scales, int scale_dtype, uint8_t* zeros,
                               bcjr_stream_t stream);

/*
 * y [tokens][rows] = x [tokens][cols] times the transpose of the 4-bit weights;
 * x and y of x_dtype, sums in float32.  float32 x is multiplied exactly (three
 * bf16 parts).  packed must be 16-byte aligned, x and y to their type, and y must
 * not overlap any of the others.  The weights are read once for every 32 tokens (10 for float32 x).
 */
bcjr_status bcjr_int4_matmul(const void* x, int x_dtype, int tokens, int rows, int cols,
                             const void* packed, const void* scales, int scale_dtype,
                             const uint8_t* zeros, int group_size, void* y, bcjr_stream_t stream);

/*
 * Trellis codes packed at k bits a weight.  A sequence's states (see
 * viterbi_decode) are windows of one bit stream: s_t is bits [t k, t k +
 * state_bits), the first bit the highest of the state and of its word, so
 * packed [n_seq][ceil((seq_len k + state_bits - k) / 32)] words hold
 * state_bits bits for the first step and k for every other.  Bits behind the
 * end are zero.  1 <= k <= 4, k <= state_bits <= 16.
 *
 * bcjr_trellis_pack packs states [n_seq][seq_len] (int32), which must be paths
 * of the trellis: when `bad` (device, one int) is given, it is set to 1 if some
 * step does not follow from the one before or a state is out of range, and left
 * as it is otherwise; the words of such a sequence are then not a path's.
 */
bcjr_status bcjr_trellis_pack(const int32_t* states, int state_bits, int k, int seq_len, int n_seq,
                              uint32_t* packed, int* bad, bcjr_stream_t stream);

/*
 * y [tokens][rows] = x [tokens][cols] times the transpose of the weights
 *   w[r][c] = codebook[state of sequence r (cols / seq_len) + c / seq_len, step c mod seq_len]
 *             * scales[c / group_size][r],
 * cols a multiple of seq_len, packed as above ([rows * cols / seq_len] sequences).
 * scales (float32 [cols / group_size][rows]) may be NULL (group_size is then
 * ignored).  group_size: 0 for one scale a row, a multiple of seq_len that
 * divides cols, or a multiple of 16 that divides seq_len.  x and y of x_dtype,
 * codebook [2^state_bits] of codebook_dtype; products and sums in float32 (by the
 * tensor core for several tokens of the codebook's own 16-bit type), the sums of
 * up to 64 columns scaled at once.  A sum of 0 under a scale that is not finite (a
 * token of zeros) is a NaN, or with 2^16 float32 codewords 0.  y must not overlap
 * any of the others.
 */
bcjr_status bcjr_trellis_matmul(const void* x, int x_dtype, int tokens, int rows, int cols,
                                const uint32_t* packed, const void* codebook, int codebook_dtype,
                                int state_bits, int k, int seq_len, const float* scales,
                                int group_size, void* y, bcjr_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* BCJR_LAYER_H */
