/*
 * lora_sample.h -- C ABI of the end of a serving step: tokens drawn from rows of logits with
 * temperature, top-k, top-p and min-p, each row with settings of its own, from given random
 * numbers.
 *
 * The conventions of lora_step.h hold: asynchronous on `stream`, no allocation, no
 * synchronisation, arguments checked on the host, device-resident settings read without a host
 * check (a row whose settings lie outside their range, or which names no row of the logits, is
 * a no-op: its outputs stay as they were), and calls may be captured and replayed.  More than
 * 2^22 - 1 rows are refused.
 */
#ifndef LORA_SAMPLE_H
#define LORA_SAMPLE_H

#include "lora_step.h"

#ifdef __cplusplus
extern "C" {
#endif

#define LORA_TYPE_F32 2                    /* logits only */
#define LORA_SAMPLE_MAX_VOCAB (1 << 22)

/*
 * One draw.  With l the row's logits (NaN counts as -inf), top their largest and t its temperature:
 *   order   tokens by logit, largest first, equal ones by index;
 *   weight  w_i = floor(2^40 exp((l_i - top) / t)), a whole number (where top is +inf: 2^40 for l_i = +inf,
 *           else 0), the exponential being right to 2^-37 of itself; masses are sums of weights, exact in
 *           64 bits, so that nothing depends on their order;
 *   top-k   the first k in order stay (k = 0: all);
 *   top-p   of these, the ones stay before which, in order, lies a mass below p times theirs; the first stays
 *           always;
 *   min-p   of these, the ones stay whose weight is at least m 2^40;
 *   token   the lowest index for which the mass of what stays up to and with it exceeds floor(u M),
 *           M being the mass of all that stays;
 *   logprob (l_token - top) / t - log(M / 2^40): its log-probability among what stays.
 * t = 0: the token of the largest logit, the lowest index among equals; logprob 0; the other
 * settings are not looked at.  A row whose logits are all -inf or NaN gets token -1 and logprob -inf.
 * Products with p, m and u are formed in 64-bit floating point.
 *
 *   logits       device [n_logits][ld] of `type`, ld >= vocab (no alignment beyond the element's)
 *   rows         device int32 [n_rows]: row of logits of each draw, or NULL (draw i reads row i)
 *   temperature  device fp32 [n_rows]: finite, >= 0; NULL: 1
 *   top_k        device int32 [n_rows]: >= 0; NULL: 0
 *   top_p        device fp32 [n_rows]: 0..1; NULL: 1
 *   min_p        device fp32 [n_rows]: 0..1; NULL: 0
 *   u            device fp32 [n_rows]: 0 <= u < 1
 *   token        device int32 [n_rows]
 *   logprob      device fp32 [n_rows] or NULL
 *   work         device memory of at least lora_sample_bytes(n_rows, vocab) bytes, 256-byte aligned, of any
 *                content; calls that may run at the same time need their own (rows fit a CU's LDS
 *                today, so its least size is all that is asked for, and it is not written)
 */
typedef struct lora_sample_args {
    int32_t type;        /* LORA_TYPE_F16, LORA_TYPE_BF16 or LORA_TYPE_F32 */
    int32_t n_rows;
    int32_t vocab;       /* 1..LORA_SAMPLE_MAX_VOCAB */
    int32_t n_logits;    /* rows of logits (>= n_rows where rows is NULL) */
    const void *logits;  int64_t ld;
    const int32_t *rows;
    const float *temperature;
    const int32_t *top_k;
    const float *top_p, *min_p, *u;
    int32_t *token;
    float *logprob;
    void *work;
    size_t work_bytes;
} lora_sample_args;

size_t lora_sample_bytes(int32_t n_rows, int32_t vocab);
int lora_sample(void *stream, const lora_sample_args *args);

#ifdef __cplusplus
}
#endif
#endif /* LORA_SAMPLE_H */
