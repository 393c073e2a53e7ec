/*
 * tpl_kv.h -- C ABI of the paged key/value cache operators for MI355X (gfx950).
 *
 * A cache is a pool of pages; a page holds the keys (and, in a second pool,
 * the values) of `page` consecutive tokens of one sequence for every key/value
 * head.  A sequence's table row names its pages in order.  A batch is packed:
 * sequence b owns rows starts[b] .. starts[b+1] of the token tensors, its
 * `lengths[b]` tokens include those new ones, and its row i stands at position
 * lengths[b] - (starts[b+1] - starts[b]) + i.
 *
 * Values are held in the tensors' own 16-bit type, or in e4m3 with one fp32
 * scale over zero for each block of `block` tokens and head: value = e4m3 *
 * scale.  (Scales under 2^-126 may count as 2^-126.)
 *
 * starts, lengths and table are read on the device only, so both calls can be
 * captured into a graph and replayed on new lengths.  Rows and pages that they
 * name outside the tensors are never touched: a table entry that is negative
 * or not a page of the pool is a page that is not there (its tokens are not
 * written, and no row sees them), and a sequence whose starts do not lie in
 * order inside the rows, that has more new tokens than its length, or more than
 * 2^30 tokens, is skipped and leaves the others as they are.  Of those others
 * each one's rows lie behind the ones before it: where they do not, rows that
 * two sequences claim, or that lie before an earlier sequence's, may be served
 * for either or not at all.
 */
#ifndef TPL_KV_H
#define TPL_KV_H

#include "tpl.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Element types. */
enum {
    TPL_KV_BF16 = 0,
    TPL_KV_FP16 = 1,
    TPL_KV_E4M3 = 2   /* OCP e4m3 (no infinities), caches only */
};

#define TPL_KV_MAX_AXES 4

/* Strides are in elements; the channels of a head are contiguous.  Every base
 * and every stride of k and v is a multiple of 16 bytes. */
typedef struct {
    void *k, *v;               /* [pages, page, kv_heads, dim] */
    float *k_scale, *v_scale;  /* [pages, kv_heads, page / block]; e4m3 only */
    int64_t pages;
    int64_t k_page, k_token, k_head;
    int64_t v_page, v_token, v_head;
    int64_t ks_page, ks_head, ks_block;
    int64_t vs_page, vs_head, vs_block;
    int32_t type;              /* TPL_KV_* of the held values */
    int32_t page;              /* tokens of a page: a multiple of 16, and of block */
    int32_t block;             /* tokens of a scale: a multiple of 16; e4m3 only */
    int32_t kv_heads, dim;     /* dim: a multiple of 16, at most 256 */
} tpl_kv_cache;

/* A batch: device arrays. */
typedef struct {
    const int32_t *table;      /* [batch, width], rows table_row apart */
    const int32_t *starts;     /* [batch + 1] */
    const int32_t *lengths;    /* [batch] */
    int64_t table_row;
    int32_t batch, width;
    int32_t tokens;            /* rows of the token tensors */
} tpl_kv_batch;

typedef struct {
    const void *k, *v;         /* [tokens, kv_heads, dim] */
    const void *q;             /* [tokens, heads, dim], or NULL */
    void *q_out;               /* q's rotated copy; may be q itself */
    const float *inv_freq;     /* [rot / 2], or NULL: no rotation */
    const int32_t *positions;  /* [axes, tokens], rows positions_row apart; NULL: a token's index in its sequence */
    int64_t k_token, k_head, v_token, v_head, q_token, q_head, o_token, o_head;
    int64_t positions_row;
    int32_t type;              /* TPL_KV_BF16 or TPL_KV_FP16: of k, v, q and q_out */
    int32_t heads;             /* of q */
    int32_t rot;               /* rotated channels: the first rot of dim, an even number */
    int32_t interleaved;       /* pairs are (2c, 2c+1); otherwise (c, c + rot/2) */
    int32_t axes;              /* 1 .. TPL_KV_MAX_AXES rows of positions */
    int32_t sections[TPL_KV_MAX_AXES]; /* axes > 1: pairs that turn by each axis, rot / 2 in all */
} tpl_kv_new;

typedef struct {
    const void *q;             /* [tokens, heads, dim] */
    void *out;                 /* [tokens, heads, dim] */
    float *lse;                /* [tokens, heads], or NULL */
    int64_t q_token, q_head, o_token, o_head, l_token, l_head;
    float scale;               /* of the scores, over zero */
    int32_t type;              /* TPL_KV_BF16 or TPL_KV_FP16: of q and out */
    int32_t heads;             /* a multiple of kv_heads */
    int32_t window;            /* 0: every earlier token; otherwise the last `window`, the row's own among them */
    int32_t sinks;             /* with a window: first tokens that stay visible */
} tpl_kv_query;

/*
 * Enqueue: rotate the new keys and queries to their positions, write keys and
 * values into their pages.
 *
 * Pair c of a head turns by position * inv_freq[c] (the angle is taken in 64
 * bits, so far positions keep their phase).  In an e4m3 cache a block's scale
 * is the least power of two, of 2^-126 at least, that brings the largest
 * finite magnitude among its new tokens (of one head, keys and values apart)
 * to 448 or under; where the block holds earlier tokens, the larger of that
 * and the scale they have, and those tokens are rounded again under it if it
 * grew.  A block's first token starts it anew: its former scale is not read.
 * Values that are not finite are held as NaN.
 */
int tpl_kv_append(const tpl_kv_cache *cache, const tpl_kv_batch *batch,
                  const tpl_kv_new *args, hipStream_t stream);

/*
 * Enqueue: out = softmax(scale * q K^T) V over the tokens each row sees, and
 * lse = the logarithm of the sum of its exponentials.  Head h of q reads head
 * h / (heads / kv_heads) of the cache.  A row that sees nothing gets zeros and
 * an lse of minus infinity.
 *
 * `workspace` is device memory of at least tpl_kv_attend_workspace() bytes,
 * 16-byte aligned.  Its first TPL_KV_COUNTERS bytes must be zero before the
 * first call that it is given to; every call leaves them zero, whichever
 * kernels it runs, so that one workspace serves any number of calls on one
 * stream.  Calls that may run at the same time need one each.
 */
#define TPL_KV_COUNTERS 4096
int tpl_kv_attend(const tpl_kv_cache *cache, const tpl_kv_batch *batch,
                  const tpl_kv_query *args, void *workspace, int64_t workspace_bytes,
                  hipStream_t stream);

/* Bytes of workspace that tpl_kv_attend needs for these sizes; -1 where it
 * would refuse the call. */
int64_t tpl_kv_attend_workspace(const tpl_kv_cache *cache, const tpl_kv_batch *batch,
                                const tpl_kv_query *args);

#ifdef __cplusplus
}
#endif

#endif /* TPL_KV_H */
