/*
 * kamera_step.h - the serving step on the paged KV pool, on AMD gfx950.
 *
 * kamera.h rebuilds cached chunks and scatters their rows into a paged pool. The calls
 * here are what a server does with that pool next, in the same library and under the same
 * conventions (kamera.h: device pointers owned by the caller, host tables read during the
 * call, a caller-supplied workspace, stream-ordered work, status codes, kamera_last_error):
 *
 *   kamera_step_upload   describe one step - the requests, their page tables, the prefixes
 *                        they share - once for all layers
 *   kamera_step_append   per layer: norm each query and key head, rotate it to its position,
 *                        write the new K and V rows into the pool's pages
 *   kamera_step_attend   per layer: attention of every query token over its request's
 *                        prefix and own tokens, a shared prefix read once for all of them
 *   kamera_copy_pages, kamera_compact_pages
 *                        copy pages inside the pool, in every layer: fork a tail page,
 *                        reorder pages, move the live pages together
 *
 * Layouts are kamera.h's. In an attention over KAMERA_MLA rows the queries are "absorbed":
 * every query head is a row of latent_dim + rope_dim columns against the one KV row of a
 * token, and the value of a token is its latent (the first latent_dim columns), so an
 * output head has latent_dim columns.
 */
#ifndef KAMERA_STEP_H_
#define KAMERA_STEP_H_

#include "kamera.h"

#ifdef __cplusplus
extern "C" {
#endif

/* step flags: what the step's plan will be launched for */
enum {
  KAMERA_STEP_APPEND = 1u, /* kamera_step_append */
  KAMERA_STEP_ATTEND = 2u, /* kamera_step_attend */
  KAMERA_STEP_FIT = 4u     /* the plan keeps to the workspace it is given (see kamera_step_workspace_bytes) */
};
/* request flags */
enum {
  KAMERA_REQUEST_ALL = 1u  /* every query sees all of the request's tokens (default: causal) */
};

/* widest key head kamera_step_attend takes (columns) */
enum { KAMERA_ATTEND_MAX_DIM = 1024 };

/* Tokens stored once and seen whole by every query of the requests that name them. */
typedef struct kamera_prefix {
  const int32_t* block_table; /* HOST page ids: token t lives at slot slot0 + t of the table       */
  int32_t slot0;              /* 0 <= slot0 < page_size                                          */
  int32_t num_tokens;         /* >= 0                                                            */
} kamera_prefix;

/* One request of a step. Its own tokens follow its prefix; the step's query tokens are the
 * last num_queries of them: query i stands at own token num_tokens - num_queries + i and
 * sees the prefix and the own tokens up to that one (KAMERA_REQUEST_ALL: all own tokens).
 * num_tokens < num_queries is allowed where nothing is appended: the first queries then see
 * the prefix alone, and without one nothing: such a row's output is 0 and its lse -inf. */
typedef struct kamera_request {
  const int32_t* block_table; /* HOST page ids of the own tokens (may be NULL if num_tokens == 0) */
  int32_t slot0;              /* 0 <= slot0 < page_size                                          */
  int32_t num_tokens;         /* own tokens >= 0, the appended ones included                     */
  int32_t num_queries;        /* >= 0; query rows of the batch are packed request after request  */
  int32_t prefix;             /* index into kamera_step.prefixes, or -1                          */
  int64_t position0;          /* rotary position of own token 0 (append; not used when
                                 kamera_step.positions is given); positions stay within 2^31     */
  uint32_t flags;             /* KAMERA_REQUEST_ALL                                              */
  int32_t reserved;           /* must be 0                                                       */
} kamera_request;

typedef struct kamera_step {
  const kamera_request* requests; /* HOST [num_requests]                                         */
  const kamera_prefix* prefixes;  /* HOST [num_prefixes]                                         */
  const int32_t* positions;       /* append: DEVICE [N][3] int32 positions (t, h, w) of the step's
                                     N query tokens, pair i of the band following the component
                                     layout.mrope_section gives it (all sections 0: t), read on
                                     `stream` by the upload; NULL: position0 + own token index    */
  int32_t num_requests;
  int32_t num_prefixes;
  int32_t num_q_heads;            /* GQA: a multiple of num_kv_heads, query head h reading KV head
                                     h / (num_q_heads / num_kv_heads); MLA: any; 0 with
                                     KAMERA_STEP_APPEND alone: no queries                          */
  uint32_t flags;                 /* KAMERA_STEP_APPEND | KAMERA_STEP_ATTEND (at least one), FIT   */
  int32_t reserved[2];            /* must be 0                                                   */
} kamera_step;

/* Written by kamera_step_upload, read by the launches; plain data, valid while the workspace
 * and the pool are untouched. */
typedef struct kamera_step_plan {
  void* workspace;
  int32_t num_tokens;   /* N: query tokens of the step */
  int32_t num_layers;
  uint32_t flags;
  int32_t reserved;
  uint64_t detail[40];
} kamera_step_plan;

/* Bytes of device workspace a step needs, whatever the pool's alignment (packed tables,
 * cos/sin of the appended tokens, partial results of the attention); 0 if the arguments are
 * invalid. They rise and fall as the lengths grow, with the number of ranges that the keys are
 * cut into. A server that allocates once asks for its largest step, with KAMERA_STEP_FIT: the
 * buffer then serves every smaller step too, that is, one made of some of the largest one's
 * requests and prefixes with at most as many tokens, queries and page-table entries each, of the
 * same layout, flags and num_q_heads. Where the fastest plan does not fit, kamera_step_upload
 * cuts the keys into fewer ranges, or lets requests read their prefix for themselves. Such a plan
 * may be slower: the largest size over the lengths that occur keeps every plan the fastest.
 * Without KAMERA_STEP_FIT a smaller workspace is refused (KAMERA_E_WORKSPACE). */
size_t kamera_step_workspace_bytes(const kamera_layout* layout, const kamera_step* step);

/* Validate a step and put its description into the workspace (256-byte aligned), on `stream`,
 * through the same staging slots as kamera_plan_upload (which see for blocking); not from a
 * capturing stream (KAMERA_E_UNSUPPORTED): record the launches of the plan instead. Pool slots that the step appends to must be distinct and must not belong to a
 * prefix of the step (KAMERA_E_OVERLAP). */
kamera_status kamera_step_upload(const kamera_layout* layout, const kamera_step* step, const kamera_pool* pool,
                                 void* workspace, size_t workspace_bytes, void* stream, kamera_step_plan* plan);

/* The new tokens of one layer. GQA: q [N][num_q_heads][head_dim], k and v [N][F]; MLA:
 * q [N][num_q_heads][F], k [N][F] (the latent and the rope band side by side), v unused.
 * A stride is in elements between tokens, 0 meaning packed, so the three may be slices of
 * one projection's rows. Element type: the layout's. q == NULL: no queries.
 *   GQA  y = x / sqrt(mean(x^2) + eps) * weight over each head's head_dim columns
 *        (weight NULL: y = x), then the rotation of the whole head.
 *   MLA  the norm covers the latent_dim columns of the KV row (q_weight must be NULL);
 *        only the rope band turns; queries' latent columns are passed on.
 * Arithmetic in fp32 (cos/sin rounded once from fp64), one rounding at the end. V rows are
 * copied. Query results go to q_out (q_out == q with equal strides: in place), K and V rows
 * to the pool slots of the step's tokens in layer `layer`. Other overlaps of what is read
 * and written are the caller's to avoid. */
typedef struct kamera_append_rows {
  const void* q;
  const void* k;
  const void* v;
  void* q_out;
  int64_t q_stride, k_stride, v_stride, q_out_stride;
  const void* q_weight; /* device [head_dim], or NULL                                   */
  const void* k_weight; /* device [head_dim] (MLA: [latent_dim]), or NULL               */
  float eps;            /* >= 0, finite                                                 */
  int32_t reserved;     /* must be 0                                                    */
} kamera_append_rows;
kamera_status kamera_step_append(const kamera_step_plan* plan, int32_t layer, const kamera_append_rows* rows,
                                 void* stream);

/* Attention of the step's N query tokens in layer `layer`:
 *     out = softmax(scale * q . K^T) V over the tokens each query sees,
 * q [N][num_q_heads][head_dim or F] (already rotated), out [N][num_q_heads][head_dim or
 * latent_dim], element type the layout's; strides in elements between tokens, 0: packed.
 * lse (fp32 [N][num_q_heads], packed, may be NULL) receives log(sum(exp(scale q.k))).
 * Scores, softmax statistics and sums are fp32; on the matrix cores the probabilities enter
 * the second product in bf16. Values of unseen tokens and unused slots are not read into any
 * result, whatever they hold. Infinities and NaN that a query sees act as in the formula (0 * inf
 * is NaN; with a scale of 0, keys that are not finite give unspecified results), but a query all
 * of whose scores are -inf has sum 0, output 0 and lse -inf. Results are the same bits on every
 * run of a step (KAMERA_STEP_FIT: in a workspace of the same size). The plan's workspace holds
 * the partial results, so launches of one plan belong on one stream at a time. */
kamera_status kamera_step_attend(const kamera_step_plan* plan, int32_t layer, const void* q, int64_t q_stride,
                                 void* out, int64_t out_stride, float* lse, float scale, void* stream);

/* In every layer, K and V: page dst[i] becomes what page src[i] was before the call, for all
 * i at once (a page may be both a source and a destination; a source may feed several).
 * src and dst are HOST arrays; the dst pages must differ (KAMERA_E_OVERLAP). The workspace
 * needs kamera_copy_pages_workspace_bytes(n) bytes, 256-byte aligned. Up to 400 copies none of
 * which writes a page that another reads travel as kernel arguments and can be recorded in a
 * captured graph; other lists are staged and cannot (KAMERA_E_UNSUPPORTED). */
size_t kamera_copy_pages_workspace_bytes(int32_t num_copies);
kamera_status kamera_copy_pages(const kamera_layout* layout, const kamera_pool* pool, const int32_t* src,
                                const int32_t* dst, int32_t num_copies, void* workspace, size_t workspace_bytes,
                                void* stream);

/* Moves the live pages - those named by the tables - together at the pool's start: with n
 * distinct live pages, those with ids >= n move, in ascending order, to the ids < n that no
 * table names, in ascending order. The HOST tables are rewritten in place (only on success)
 * and *num_live receives n. A page named several times (shared) moves once, and tables may be
 * parts of one array, the same parts among them. The workspace
 * needs kamera_copy_pages_workspace_bytes(pages that move) bytes; their number is at most n. */
kamera_status kamera_compact_pages(const kamera_layout* layout, const kamera_pool* pool, int32_t* const* tables,
                                   const int32_t* lengths, int32_t num_tables, int32_t* num_live, void* workspace,
                                   size_t workspace_bytes, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* KAMERA_STEP_H_ */
