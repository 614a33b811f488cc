/*
 * lora_quant.h -- C ABI of a paged key/value cache held in 4 or 8 bits: the append that
 * quantises what it writes, reading cells back, and attention over the cache.  The operators
 * stand beside those of lora_step.h, whose plan, tables, slots and rotary positions they
 * take; a layer uses either cache.
 *
 * The conventions of lora_step.h hold (pointers to codes and to 16-bit data are 16-byte
 * aligned; exponents are bytes of any alignment).  lora_quant_append and lora_quant_read take
 * any number of rows below 2^24 - 128, and may refuse more.
 *
 * The format.  The head_dim columns of one token and head are cut into blocks of 32 (the
 * last one padded with zeros).  A block is 32 codes and one exponent byte e; code c stands for
 *     c * 2^(e - 127),
 * and a block with e = 255 for 32 NaN.  Codes of 4 bits are E2M1 (0, 0.5, 1, 1.5, 2, 3, 4, 6,
 * and their negatives with bit 3 set; the first of two columns in the low half of its byte), codes of 8
 * bits E4M3 (largest value 448, no infinities).  A cache has a 16-bit type, and the exponents
 * written are kept to what that type holds:
 *                          4 bits             8 bits
 *     LORA_TYPE_F16     e - 127 in -23..13      -15..7
 *     LORA_TYPE_BF16            -125..125      -117..119
 * so every value of a cell that was appended is a value of the 16-bit type exactly: reading
 * rounds nothing.  Where something else has written a cell, its exponent may be any byte (e = 0 is
 * the power 2^-127): a value that the type does not hold is rounded to it wherever the cell is
 * read, to nearest, ties to even, as far as to 0 and to infinity.
 *
 * Quantising a block: e - 127 is the smallest power with max|x| < 7 * 2^(e-127) (4 bits; no
 * element is then off by more than 2^(e-127), half of the largest step), or with max|x| <
 * 464 * 2^(e-127) (8 bits; half of a step above 448), kept to the range above; codes are
 * x * 2^(127-e) rounded to nearest, ties to even, and what lies beyond the largest code takes
 * it (only where the range above cut e off).  A block with an infinity or a NaN gets e = 255.
 */
#ifndef LORA_QUANT_H
#define LORA_QUANT_H

#include "lora_step.h"

#ifdef __cplusplus
extern "C" {
#endif

#define LORA_QUANT_BLOCK 32

/*
 * One layer's cache.  Token `off` of page p and head h: head_dim columns, padded to `blocks` =
 * ceil(head_dim / 32) blocks, whose codes are the 4 * bits * blocks contiguous bytes at
 *     k + p*page_stride + off*token_stride + h*head_stride                (v alike)
 * and whose exponents are the `blocks` bytes at
 *     k_exp + p*exp_page_stride + off*exp_token_stride + h*exp_head_stride   (v_exp alike).
 * Heads before tokens in memory ([page][head][token]) keeps the tokens that one head reads
 * together, which is what the attention runs fastest on.  The tokens of one page and head span
 * less than 2^31 bytes; everything else may lie 2^48 bytes apart.  The slot of a token is
 * p*page_size + off; num_pages * page_size <= 2^31 - 1.  Memory of zeros reads as zeros.
 * Codes of columns from head_dim on are written as 0 and take no part in any result, but a
 * block's exponent byte is shared: they must not be NaN (8 bits: 0x7f, 0xff) in a cache that
 * something else has written.
 */
typedef struct lora_quant_cache {
    int32_t type;        /* LORA_TYPE_*: of the values, and of every 16-bit argument of a call */
    int32_t bits;        /* 4 or 8 */
    int32_t page_size;   /* tokens per page: a power of two, 1..LORA_KV_MAX_PAGE */
    int32_t num_pages;   /* >= 1 */
    int32_t kv_heads;    /* >= 1 */
    int32_t head_dim;    /* a multiple of 8, 8..LORA_KV_MAX_HEAD_DIM */
    int64_t page_stride, token_stride, head_stride; /* bytes, multiples of 16, >= 4 * bits * blocks (even where a size is 1) */
    int64_t exp_page_stride, exp_token_stride, exp_head_stride; /* bytes, >= blocks (even where a size is 1) */
    void *k, *v;             /* device, 16-byte aligned */
    uint8_t *k_exp, *v_exp;  /* device */
} lora_quant_cache;

/*
 * lora_rope_append into a quantised cache: for every token row t with slots[t] in
 * [0, num_pages * page_size):
 *     q_out[t] = rotated q[t],
 *     the cells of k at slots[t] = rotated k[t], of v = v[t], quantised.
 * k is rotated in 64 bits, rounded to 32 and quantised from there.  Everything else is as
 * in lora_rope_append: rows with another slot leave q_out and the cache as they were; q_out
 * may be q itself; two rows of one call must not name the same slot.
 */
int lora_quant_append(void *stream, int32_t n_rows, int32_t q_heads, void *q_out, int64_t ldqo, const void *q,
                      int64_t ldq, const void *k, int64_t ldk, const void *v, int64_t ldv, const lora_rope *rope,
                      const int32_t *positions, int64_t ld_pos, const int32_t *slots, const lora_quant_cache *cache);

/*
 * Reads cells back: for every row t with slots[t] in [0, num_pages * page_size), k_out[t] and
 * v_out[t] (kv_heads heads of head_dim elements of the cache's type) take the values of
 * that token's cells; other rows stay as they were.  k_out or v_out may be NULL.  Any slots, repeated ones too.
 *   k_out, v_out  device [n_rows][ld], ld % 8 == 0, ld >= kv_heads * head_dim; they share no
 *                 element with each other
 */
int lora_quant_read(void *stream, int32_t n_rows, void *k_out, int64_t ldko, void *v_out, int64_t ldvo,
                    const int32_t *slots, const lora_quant_cache *cache);

/*
 * lora_paged_attention over a quantised cache: the same arguments, rows, masks and results
 * with k_t and v_t the values of the cells, as lora_quant_read gives them.  The products are those of
 * the exact values; softmax weights multiply v as two 16-bit parts, as there (fp16: a weight below
 * 2^-38 of the row's largest counts as 0).  A visible NaN makes its row's head NaN, and a
 * visible infinity (appended cells hold none) may.  n_rows times the tiles of the longest row, here 64
 * tokens each and eight more a row, stays 2048 below 2^31, or the call is refused.
 *   work   device memory of at least lora_quant_attention_bytes(...) bytes, 256-byte aligned,
 *          all zero before its first use; every call leaves its counters zero again.  Calls
 *          ordered on one stream (graph replays included) may share it, with
 *          lora_paged_attention too; calls that may run at the same time need their own.
 */
size_t lora_quant_attention_bytes(int32_t n_rows, int32_t q_heads, int32_t kv_heads, int32_t head_dim);
int lora_quant_attention(void *stream, int32_t n_rows, int32_t q_heads, void *out, int64_t ldo, const void *q,
                         int64_t ldq, const lora_quant_cache *cache, int32_t n_req, const int32_t *block_table,
                         int64_t ld_table, int32_t max_blocks, const int32_t *kv_len, const int32_t *req, float scale,
                         int32_t window, float *lse, void *work, size_t work_bytes);

#ifdef __cplusplus
}
#endif
#endif /* LORA_QUANT_H */
