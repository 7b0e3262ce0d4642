/*
 * gkd_blocks.h - C ABI of libgkd, continued: the operators of the transformer
 * blocks around the detection head (gkd.h). In GKDT the prompt rows that the
 * head uses as kernels come out of such blocks, and so do the features they are
 * matched against.
 *
 * Sources (titles and sections of the pages that name the blocks):
 *   [CARD]  Asher-1/GKD_GGUF model card, section Model, Architecture bullet: a
 *           vision tower (width 1024, 24 blocks, 16 heads) with rotary positions,
 *           layer scale and extra storage and class tokens beside the patches; a
 *           text tower (width 1280, 24 causal blocks, 20 heads); a linear text
 *           head from 1280 to 2048; an adaptation net with QuickGELU; a kernel
 *           generator of 2 blocks with self- and cross-attention and a
 *           feed-forward width of 1024; prompts padded to 80 rows under a mask.
 *           Conversion notes: the rotary periods are exported from the checkpoint.
 *   [NOTES] GKDT reading notes, section Method: the prototypes attend to one
 *           another and to the query before they become kernels.
 *
 * The conventions of gkd.h hold: device pointers owned by the caller, host-side
 * validation before any launch, work enqueued on `stream` on the device of the
 * first tensor argument, no allocation, no synchronisation, gkd_status codes,
 * gkd_last_error(), 16-byte alignment of tensor base pointers and byte strides.
 * A call whose outputs would be empty returns GKD_OK and launches nothing.
 * Waits inside the kernels have gkd.h's limit (gkd_set_wait_timeout_ms) and report to
 * its error word (gkd_check_device_error).
 * Outputs may be used on another stream once that stream waits for `stream`.
 * No call keeps state between calls: calls may run at once on any streams, and
 * captured calls may be replayed in any order. Results do not depend on
 * scheduling (every sum has a fixed order).
 */
#ifndef GKD_BLOCKS_H_
#define GKD_BLOCKS_H_

#include "gkd.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef enum gkd_activation {
  GKD_ACT_NONE = 0,
  GKD_ACT_RELU = 1,
  GKD_ACT_GELU = 2,        /* y Phi(y), Phi the normal distribution function (erf) */
  GKD_ACT_QUICK_GELU = 3   /* y / (1 + exp(-1.702 y)) */
} gkd_activation;

/*
 * Heads of a batch of rows: element (b, t, h, i) of [B][rows][heads][D] lies at
 * data + b * batch_stride + t * row_stride + h * head_stride + i. Any layout whose
 * last axis is contiguous has such strides: [B][rows][heads][D], [B][heads][rows][D],
 * a slice of a buffer that holds queries, keys and values side by side. Strides of
 * axes of size 1 are not looked at. An input may have batch_stride 0 (one tensor
 * shared by the whole batch).
 */
typedef struct gkd_heads {
  void* data;
  long long batch_stride, row_stride, head_stride;   /* in elements */
  int heads;
} gkd_heads;

/*
 * Linear layer with its epilogue ([CARD] Architecture bullet: text head,
 * feed-forwards, QuickGELU, layer scale):
 *
 *   out[t,n] = residual[t,n] + scale[n] * act(sum_c x[t,c] * weight[n,c] + bias[n])
 *
 *   x         [T][Cin], rows x_stride apart; dt = GKD_BF16 or GKD_F32
 *   weight    [Cout][Cin] of type dt, contiguous
 *   bias      [Cout] fp32, or NULL (0)
 *   scale     [Cout] fp32, or NULL (1)
 *   residual  [T][Cout] of type out_dt, rows residual_stride apart, or NULL (0).
 *             It may be `out` itself (with the same stride), and must not overlap it
 *             otherwise.
 *   out       [T][Cout], rows out_stride apart, out_dt = GKD_BF16 or GKD_F32
 *             (dt = GKD_F32 takes GKD_F32 only). Columns past Cout are left alone.
 * dt = GKD_BF16: exact products, sums in fp32 (for an fp32 output at most 512 channels
 * at a time on the tensor core, whose sums truncate). dt = GKD_F32: every operand as a
 * pair of TF32 numbers, three products per term, each term within 2^-19 of its product
 * (on average 1.5e-7 short of it); x and weight must be finite (an infinity gives NaN
 * or an infinity in its own row or column). The epilogue is in
 * fp32, with one rounding to out_dt. `out` must not overlap x or weight.
 * Limits: 0 <= T < 2^31, 8 <= Cin, Cout <= 65536, both multiples of 8, strides
 * at least the row's length.
 */
GKD_API gkd_status gkd_linear(const void* x, gkd_dtype dt, int T, int Cin, long long x_stride, const void* weight,
                              int Cout, const float* bias, gkd_activation act, const float* scale,
                              const void* residual, long long residual_stride, void* out, gkd_dtype out_dt,
                              long long out_stride, void* stream);

/*
 * Norms of the query and key heads and their rotation by position, in one pass
 * ([CARD] Architecture bullet and conversion notes: rotary positions with the
 * checkpoint's periods). For every row t of every head of q, and of k:
 *
 *   y     = x * weight / sqrt(mean_i x_i^2 + eps)          (weight NULL: y = x)
 *   angle = pos[t, pair_axis[p]] * pair_freq[p]              for pairs p < pairs
 *   (y_a, y_b) -> (y_a cos - y_b sin, y_b cos + y_a sin)     (a, b) = (p, p + pairs), or
 *                                                            (2 p, 2 p + 1) if interleaved
 * and the elements from 2 * pairs on keep y. A row whose positions are 0 (class and
 * storage tokens) is not turned.
 *
 *   q, k        [B][T] rows of q->heads and k->heads heads of D elements, type dt.
 *               k may be NULL (queries alone; k_out is then NULL too).
 *   q_weight, k_weight   [D] fp32, or both NULL (no norm; eps is not looked at)
 *   pos         [T][axes] fp32; batch b's at pos + b * pos_batch_stride (0 = shared)
 *   pair_axis   [pairs] uint8, the axis that turns each pair. Values >= axes are
 *               taken as axis 0.
 *   pair_freq   [pairs] fp32, radians per unit of position
 *   q_out, k_out  as q and k (the same head counts). Each may be its input itself,
 *               with the same strides, and must not overlap anything else of the call
 *               (q_out not k, k_out not q, nor one the other).
 * Angles are formed and reduced in fp64 (positions up to 2^24 keep fp32 accuracy),
 * everything else in fp32, rounded once to dt.
 * Limits: 0 <= B <= 65535, 0 <= T < 2^31, 8 <= D <= 256, D % 8 == 0, 1 <= heads <= 1024,
 * 1 <= axes <= 3, 0 <= pairs <= D / 2, pairs % 4 == 0, eps > 0 with weights. With
 * pairs == 0 pos, pair_axis and pair_freq are not looked at.
 */
GKD_API gkd_status gkd_qk_norm_rope(const gkd_heads* q, const gkd_heads* k, gkd_dtype dt, int B, int T, int D,
                                    const float* q_weight, const float* k_weight, float eps, const float* pos,
                                    long long pos_batch_stride, int axes, const uint8_t* pair_axis,
                                    const float* pair_freq, int pairs, int interleaved, const gkd_heads* q_out,
                                    const gkd_heads* k_out, void* stream);

/*
 * Attention under a key mask ([CARD] Architecture bullet and [NOTES] Method: the
 * kernel generator's self- and cross-attention over padded prompt rows, the
 * towers' self-attention, causal in the text tower):
 *
 *   out[b,i,h,:] = sum_j p_j v[b,j,g,:] / sum_j p_j,
 *   p_j = exp(scale * q[b,i,h,:] . k[b,j,g,:] - max_j'(...)),   g = h * k->heads / q->heads
 * over the keys j with key_mask[b,j] != 0 (all, if NULL) and, if causal,
 * j <= i + Tk - Tq (the last query sees every key). Rows without such a key are 0.
 * Keys and values that the key mask hides may hold anything, NaN included. A NaN or an
 * infinity in a value v[b,j] that the mask does not hide can reach any row of its batch
 * and head, also one that the diagonal keeps from key j.
 *
 *   q        [B][Tq] rows of q->heads heads of D elements, type dt
 *   k, v     [B][Tk] rows; k->heads == v->heads divides q->heads
 *   key_mask uint8, batch b's [Tk] at key_mask + b * key_mask_batch_stride (0 = shared), or NULL
 *   out      as q. It must not overlap the inputs.
 * dt = GKD_BF16: tensor-core products with fp32 accumulation; maxima, sums and
 * exponentials in fp32; the weights p_j are rounded to bf16 for the product with v
 * (their sum is not). dt = GKD_F32: every operand as three bf16 numbers (24 bits), six
 * products per term, the rest in fp32 (up to 24 keys or 12 queries, and 16 where that is
 * faster: fp32 fused multiply-adds); visible q, k and v must be finite and below 2^127 in magnitude (others
 * can give NaN, and so can scores that overflow). The sum of p_j v is formed before its
 * division: values of one sign above 2^127 / Tk (bf16: 2^119 / Tk) can overflow in it,
 * and above 2^55 / Tk where scale * score passes 2^24 (the rounding of the largest one
 * is common to a row's weights, and 2^64 at most).
 * A score of -inf has weight 0 beside larger ones. A row with a score of NaN or +inf is
 * NaN, and so is one whose scores are all -inf.
 * Limits: 0 <= B <= 65535, 0 <= Tq, Tk < 2^31 - 256, 8 <= D <= 128, D % 8 == 0,
 * 1 <= heads <= 1024, 0 < scale < 2^127.
 */
GKD_API gkd_status gkd_attention(const gkd_heads* q, const gkd_heads* k, const gkd_heads* v, gkd_dtype dt, int B,
                                 int Tq, int Tk, int D, float scale, int causal, const uint8_t* key_mask,
                                 long long key_mask_batch_stride, const gkd_heads* out, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* GKD_BLOCKS_H_ */
