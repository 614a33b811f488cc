/*
 * lora_step.h -- C ABI of the decode-step operators beside the multi-LoRA add-on
 * (lora_sgmv.h): the step's page and token maps, rotary positions with the append to a
 * paged key/value cache, attention over that cache, and the residual add with its norms.
 *
 * One serving step runs, per batch, lora_kv_plan, and per layer lora_residual_norm, the
 * q/k/v projections with their add-ons, lora_rope_append, lora_paged_attention, the
 * output projection, lora_residual_norm, and the feed-forward part.
 *
 * The conventions of lora_sgmv.h hold: the caller owns every buffer; calls are
 * asynchronous on `stream`, allocate nothing, never synchronise and keep no state; all
 * device pointers to 16-bit data are 16-byte aligned (lse, inv_freq and the int32 arrays 4);
 * arguments are checked on the host before any launch, and LORA_OK or a negative LORA_E_*
 * code is returned (lora_last_error() describes it).  Device-resident metadata (lengths, slots,
 * page ids) is read without a host check, and an entry outside its documented range
 * makes its row, token or page a no-op instead of an out-of-bounds access.  Every call
 * may be captured into a graph and replayed with new metadata in the same arrays.  The
 * diagnostics of lora_sgmv.h (launch events, plans) apply to the add-on's launches only.
 * A launch has at most 2^32 - 1 threads: the calls with a workgroup of 64 to 1024 threads
 * per row (lora_rope_append, lora_residual_norm) refuse more rows than that holds, which is
 * never fewer than 2^22 - 1.
 *
 * Types: `type` is LORA_TYPE_F16 (IEEE binary16) or LORA_TYPE_BF16 for all 16-bit data
 * of a call.  Arithmetic is fp32 (sums, softmax statistics, norms), angles are 64-bit;
 * each output is rounded once (to nearest even).  Results are bit-identical from run to
 * run for the same inputs.
 */
#ifndef LORA_STEP_H
#define LORA_STEP_H

#include "lora_sgmv.h"

#ifdef __cplusplus
extern "C" {
#endif

#define LORA_TYPE_F16 0
#define LORA_TYPE_BF16 1

#define LORA_KV_MAX_PAGE 1024     /* largest page, in tokens */
#define LORA_KV_MAX_HEAD_DIM 256  /* largest head dimension */
#define LORA_ROPE_MAX_AXES 4      /* position axes of one rotary embedding */
#define LORA_NORM_MAX_HIDDEN 65536

/* ---------------------------------------------------------------- the paged cache */
/*
 * One layer's key/value cache (S-LoRA summary, "Unified Paging": the cache is held in
 * pages of one pool, found through a table).  Token `off` of page p and head h is the
 * head_dim contiguous elements at
 *     k + p*page_stride + off*token_stride + h*head_stride     (v alike)
 * so [page][token][head][dim] and [page][head][token][dim] are both covered.  The slot
 * of a token is p*page_size + off.  num_pages * page_size <= 2^31 - 1; byte offsets are
 * 64-bit.
 */
typedef struct lora_kv_cache {
    int32_t type;        /* LORA_TYPE_* */
    int32_t page_size;   /* tokens per page: a power of two, 1..LORA_KV_MAX_PAGE */
    int32_t num_pages;   /* >= 1 */
    int32_t kv_heads;    /* >= 1 */
    int32_t head_dim;    /* a multiple of 8, 8..LORA_KV_MAX_HEAD_DIM */
    int32_t reserved;    /* 0 */
    int64_t page_stride, token_stride, head_stride; /* elements, multiples of 8, >= head_dim (> 0 even where a size is 1) */
    void *k, *v;         /* device */
} lora_kv_cache;

/* ---------------------------------------------------------------- step plan */
/*
 * Block tables and the free-page list of a batch's requests, on the device.  Row r of
 * block_table holds the pages of request r in token order; entries from
 * ceil(kv_len[r] / page_size) on are not read.  free_pages is a stack: entries
 * [0, *free_top) are the free ids, the last one is taken first.
 */
typedef struct lora_kv_pages {
    int32_t n_req;         /* rows of the batch's tables: 0..2^30 */
    int32_t page_size;     /* a power of two, 1..LORA_KV_MAX_PAGE */
    int32_t num_pages;     /* capacity of free_pages (>= 1) */
    int32_t max_blocks;    /* entries of a table row (>= 1); max_blocks * page_size <= 2^31 - 1 */
    int64_t ld_table;      /* >= max_blocks */
    int32_t *block_table;  /* device [n_req][ld_table], updated in place */
    int32_t *free_pages;   /* device [num_pages], updated in place */
    const int32_t *free_top; /* device [1]: 0..num_pages */
} lora_kv_pages;

/* What a plan writes; every array is device memory. */
typedef struct lora_kv_plan_out {
    int32_t max_tokens;    /* rows of the token maps (>= 0) */
    int32_t reserved;      /* 0 */
    int32_t *status;       /* [4]: LORA_KV_* bits (0 = planned); tokens; pages taken; pages returned */
    int32_t *kv_end;       /* [n_req]: cached tokens after the step; may be kv_len itself */
    int32_t *free_top;     /* [1]: free pages after the step; may be pages->free_top itself */
    int32_t *q_ptr;        /* [n_req + 1]: first token row of each request (lora_segments.seg_ptr of the step) */
    int32_t *tok_req;      /* [max_tokens]: request of each token row, -1 behind the last token */
    int32_t *tok_pos;      /* [max_tokens]: position in its request, -1 behind the last token */
    int32_t *slots;        /* [max_tokens]: cache slot, -1 behind the last token */
    int32_t *idx;          /* [max_tokens] or NULL: adapter slot of each token row (req_slot of its
                              request; -1 behind the last token): the idx of the per-row add-on calls */
} lora_kv_plan_out;

#define LORA_KV_NO_PAGES 1   /* fewer free pages than the step takes */
#define LORA_KV_TOO_LONG 2   /* a request outgrows its table row */
#define LORA_KV_TOO_MANY 4   /* more new tokens than max_tokens */
#define LORA_KV_INVALID 8    /* kv_len < 0, new_len < -1, *free_top outside 0..num_pages, or more
                                pages returned than the list can hold */

/*
 * Plans one step on the device from the requests' lengths (Punica summary, "Batch Layout
 * Construction": the batch's metadata is built once per step and reused by every layer).
 *   kv_len  device int32 [n_req]: tokens each request has in the cache (>= 0)
 *   new_len device int32 [n_req]: tokens it adds in this step (>= 0); -1: the request has
 *           ended, its ceil(kv_len / page_size) pages go back to the free list and its
 *           kv_end is 0
 *   req_slot device int32 [n_req] or NULL: adapter slot of each request (out->idx)
 * Pages of ended requests are put on the free list first, in request and table order;
 * then the growing requests take ceil((kv_len + new_len) / page_size) -
 * ceil(kv_len / page_size) pages each from its end, in request order, which become their
 * table entries.  Token rows are numbered in request order: row q_ptr[r] + i is token
 * kv_len[r] + i of request r.
 * All or nothing: if any LORA_KV_* bit is set, the tables and the free list stay as they
 * were, kv_end = kv_len, the free top is copied, q_ptr is all 0 and the maps are all -1
 * (the step's other calls then do nothing); status[1..3] still give what the step asked
 * for (clamped to 2^31 - 1).  Page ids are moved, never followed.  The arrays written share
 * no entry with each other or with those read, other than kv_end and free_top as said.
 * Two plans of one free list or table must be ordered on one stream.
 */
int lora_kv_plan(void *stream, const lora_kv_pages *pages, const int32_t *kv_len, const int32_t *new_len,
                 const int32_t *req_slot, const lora_kv_plan_out *out);

/* ---------------------------------------------------------------- rotary positions and append */
/*
 * Rotary positions with one or several axes (text; or time, height and width of an
 * image or video token).  Frequency i (0 <= i < rot_dim/2) turns one pair of elements of
 * every head by the angle position[axis[i]] * inv_freq[i]:
 *     (a, b) -> (a cos - b sin, a sin + b cos)
 * where the pair is (x[i], x[i + rot_dim/2]), or (x[2i], x[2i + 1]) with `interleaved`.
 * Elements from rot_dim on pass through.  Angles are formed and reduced in 64 bits, so
 * far positions keep their precision.
 */
typedef struct lora_rope {
    int32_t rot_dim;        /* a multiple of 16, 0..head_dim (0: append without rotation) */
    int32_t n_axes;         /* 1..LORA_ROPE_MAX_AXES */
    int32_t interleaved;    /* 0 or 1 */
    int32_t reserved;       /* 0 */
    const float *inv_freq;  /* device [rot_dim/2]; NULL allowed when rot_dim is 0 */
    const int32_t *axis;    /* device [rot_dim/2] or NULL (all on axis 0); a frequency whose axis is
                               outside 0..n_axes-1 is not turned */
} lora_rope;

/*
 * For every token row t with slots[t] in [0, num_pages * page_size):
 *     q_out[t] = rotated q[t]   (q_heads heads of head_dim),
 *     cache k at slots[t] = rotated k[t], cache v at slots[t] = v[t].
 * Rows with another slot (-1: no token) leave q_out and the cache as they were.
 * q, k, v: device [n_rows][ld*], ld % 8 == 0 (column slices of one product are fine);
 * q_out may be q itself (same leading dimension), and must not overlap the inputs
 * otherwise; none of the four may overlap the cache.  q and q_out may both be NULL with
 * q_heads 0.  positions: device int32 [n_axes][ld_pos], ld_pos >= n_rows (NULL allowed when
 * rot_dim is 0).  Two rows of one call must not name the same slot.
 */
int lora_rope_append(void *stream, int32_t n_rows, int32_t q_heads, void *q_out, int64_t ldqo, const void *q,
                     int64_t ldq, const void *k, int64_t ldk, const void *v, int64_t ldv, const lora_rope *rope,
                     const int32_t *positions, int64_t ld_pos, const int32_t *slots, const lora_kv_cache *cache);

/* ---------------------------------------------------------------- attention over the paged cache */
/*
 * One query token per row: for row i with r = req ? req[i] : i and n = kv_len[i], head h
 * of q_heads and its key/value head g = h / (q_heads / kv_heads),
 *     s_t = scale * <q[i][h], k_t>        for the tokens t of request r with t < n and,
 *                                         with window > 0, t >= n - window,
 *     out[i][h] = sum_t exp(s_t - m) v_t / sum_t exp(s_t - m),   m = max_t s_t,
 *     lse[i][h] = m + log(sum_t exp(s_t - m)).
 * Token t lies in page block_table[r][t / page_size].  Tokens of a page id outside
 * [0, num_pages) are left out, and values at positions that are left out are never
 * used (stale infinities and NaN there do not matter).  A row with nothing left (n = 0,
 * or every s_t = -inf) gets out = 0 and lse = -inf.  Rows with n < 0, n > max_blocks *
 * page_size or r outside [0, n_req) are not active: out and lse stay as they were there.
 * Several rows may name one request (each with its own n), e.g. the tokens of a guess
 * that is being verified; each row reads its tokens for itself.
 * Softmax weights multiply v as two 16-bit parts: bf16 keeps 16 bits of a weight, fp16 22 bits
 * and never less than 2^-37 of the row's largest one, so that beside the rounding of the
 * output, n visible tokens put an fp16 row off by up to n 2^-37 max_t |v_t| (half an fp16
 * step of that maximum at n = 2^26).
 * n_rows times the tiles of the longest row that max_blocks (or the window) allows, 32 tokens
 * each and four more a row, stays 512 below 2^31, or the call is refused
 * (LORA_E_UNSUPPORTED): 63 rows at 2^30 tokens, 65,000 at 2^20.
 *
 *   out, q       device [n_rows][ld], ld % 8 == 0, ld >= q_heads * head_dim; the cache's type
 *   q_heads      a multiple of kv_heads
 *   block_table  device int32 [n_req][ld_table], ld_table >= max_blocks;
 *                max_blocks * page_size <= 2^30
 *   kv_len       device int32 [n_rows] (the query's own token included)
 *   req          device int32 [n_rows] or NULL
 *   scale        any finite value (usually 1/sqrt(head_dim))
 *   window       0 (none) or the number of last tokens a row sees
 *   lse          device fp32 [n_rows][q_heads] or NULL
 *   work         device memory of at least lora_paged_attention_bytes(...) bytes, 256-byte
 *                aligned, all zero before its first use; every call leaves its counters
 *                zero again.  Calls ordered on one stream (graph replays included) may
 *                share it; calls that may run at the same time need their own.
 */
size_t lora_paged_attention_bytes(int32_t n_rows, int32_t q_heads, int32_t kv_heads, int32_t head_dim);
int lora_paged_attention(void *stream, int32_t n_rows, int32_t q_heads, void *out, int64_t ldo, const void *q,
                         int64_t ldq, const lora_kv_cache *cache, int32_t n_req, const int32_t *block_table,
                         int64_t ld_table, int32_t max_blocks, const int32_t *kv_len, const int32_t *req, float scale,
                         int32_t window, float *lse, void *work, size_t work_bytes);

/* ---------------------------------------------------------------- residual add and norms */
/*
 * Around a block of the layer, for every row i (hidden elements; all products per element):
 *     p = post_w ? rms(x[i]) * (post_w + w_offset) : x[i]         (norm after the block)
 *     h = res[i] + alpha * gate_i * p
 *     res_out[i] = h,   y[i] = rms(h) * (w + w_offset)            (norm before the next block)
 * with rms(z) = z / sqrt(mean(z^2) + eps).  y is normed from h before h is rounded.
 * gate_i: row gate_idx[i] of gate [n_gates][hidden]; all ones where gate is NULL or
 * gate_idx[i] is -1; row 0 for every i where gate_idx is NULL (n_gates is then 1).  A
 * gate_idx outside [-1, n_gates) makes its row a no-op.
 *   x        NULL: nothing is added (h = res; post_w and gate must be NULL too)
 *   res_out  NULL: not written; may be res itself
 *   y        NULL: not written (w is then not read); may be x itself
 *   w, post_w, gate  of the call's type; w_offset is added to w and post_w (0, or 1 for
 *            weights stored as an offset from one)
 * hidden: a multiple of 8, 8..LORA_NORM_MAX_HIDDEN.  ld % 8 == 0.  Outputs must not
 * overlap inputs other than as said.
 */
typedef struct lora_norm_args {
    int32_t type, n_rows, hidden, n_gates;
    void *y;              int64_t ldy;
    void *res_out;        int64_t ldro;
    const void *res;      int64_t ldr;
    const void *x;        int64_t ldx;
    const void *w;        /* device [hidden] */
    const void *post_w;   /* device [hidden] or NULL */
    const void *gate;     int64_t ldg;
    const int32_t *gate_idx; /* device [n_rows] or NULL */
    float alpha, eps, w_offset;
    int32_t reserved;     /* 0 */
} lora_norm_args;

int lora_residual_norm(void *stream, const lora_norm_args *args);

#ifdef __cplusplus
}
#endif
#endif /* LORA_STEP_H */
