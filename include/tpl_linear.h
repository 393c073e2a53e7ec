/*
 * tpl_linear.h -- C ABI of linear attention with a decay for each head, for
 * MI355X (gfx950).
 *
 * A layer's past is one state a head, [key_dim, value_dim] in fp32, instead of
 * keys and values of every token.  A pool holds such states in slots.  For each
 * of a sequence's new tokens in order
 *
 *     S = exp(decay) S + k v^T        out = scale * q S
 *
 * A batch is packed as those of tpl_kv.h are: sequence b owns rows starts[b] ..
 * starts[b+1] of the token tensors.  Its state before them is what slot
 * sources[b] holds, and zero where that is not a slot of the pool; the state
 * after them is written to slot slots[b], and to none where that is not one.
 * So a sequence goes on in place (both name one slot), begins (source -1), or
 * forks (a slot of its own).  A slot that a call writes is written by one
 * sequence and read by no other.  A sequence without rows, or whose starts do
 * not lie in order inside the rows, is skipped and leaves the others, its rows
 * and its slots as they are.  Of the others each one's rows lie behind the ones
 * before it: rows that two claim may be served for either or not at all.
 *
 * slots, sources, starts and the decays are read on the device only, so that a
 * call can be captured into a graph and replayed on new numbers.
 */
#ifndef TPL_LINEAR_H
#define TPL_LINEAR_H

#include "tpl_kv.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Strides are in elements; a state's value channels and a head's channels are
 * contiguous.  Every base and stride lies on 16 bytes; rows of q, k and v lie
 * under 2^24 elements apart. */
typedef struct {
    float *state;              /* [slots, heads, key_dim, value_dim] */
    const float *decay;        /* [heads]: logarithms; what is over zero counts as zero */
    int64_t s_slot, s_head, s_key;
    int64_t slots;
    int32_t heads, key_dim, value_dim;   /* dims: multiples of 16, at most 256 */
} tpl_linear_pool;

/* Device arrays. */
typedef struct {
    const int32_t *slots;      /* [batch] */
    const int32_t *sources;    /* [batch], or NULL: slots */
    const int32_t *starts;     /* [batch + 1] */
    int32_t batch;
    int32_t tokens;            /* rows of the token tensors */
} tpl_linear_batch;

typedef struct {
    const void *q, *k;         /* [tokens, key_heads, key_dim] */
    const void *v;             /* [tokens, heads, value_dim] */
    void *out;                 /* [tokens, heads, value_dim]; not over q or k */
    int64_t q_token, q_head, k_token, k_head, v_token, v_head, o_token, o_head;
    float scale;               /* a finite number */
    int32_t type;              /* TPL_KV_BF16 or TPL_KV_FP16: of q, k, v and out */
    int32_t key_heads;         /* divides heads: head h reads q and k of head h / (heads / key_heads) */
} tpl_linear_new;

/*
 * Enqueue the above.  States, sums and products are held in fp32 (16-bit
 * products of the parts of fp32 numbers, two parts each); out is rounded once.
 *
 * `workspace`: device memory of at least tpl_linear_attend_workspace() bytes,
 * 16-byte aligned, of any contents; calls that may run at the same time need
 * one each.
 */
int tpl_linear_attend(const tpl_linear_pool *pool, const tpl_linear_batch *batch,
                      const tpl_linear_new *args, void *workspace, int64_t workspace_bytes,
                      hipStream_t stream);

/* Bytes of workspace that tpl_linear_attend needs for these sizes; -1 where it
 * would refuse the call. */
int64_t tpl_linear_attend_workspace(const tpl_linear_pool *pool, const tpl_linear_batch *batch,
                                    const tpl_linear_new *args);

#ifdef __cplusplus
}
#endif

#endif /* TPL_LINEAR_H */
