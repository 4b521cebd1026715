/*
 * libkda -- latent attention for serving, on one NVIDIA GB300 (sm_103a): the
 * full-attention layers that models interleave with KDA layers, in the form
 * that keeps ONE shared latent vector a token in a paged cache.
 *
 * A cache row (one token) is 512 latent values c followed by 64 key values
 * k_pe that all heads share, bf16.  Four calls cover a serving step:
 *
 *   kda_latent_plan     block tables and slot maps on the GPU from request lengths
 *   kda_latent_append   new tokens' rows (latents optionally RMS-normalised)
 *                       into the cache through the slot map
 *   kda_latent_decode   absorbed form: query heads live in the latent space,
 *                         s = scale q . [c | k_pe],  o = softmax(s) c
 *                       one or a few new tokens a request against the cache
 *   kda_latent_prefill  expanded form: per-head keys [k (128) | k_pe (64)] and
 *                       values v (128), prompts dense or packed
 *
 * With k_h = W_uk,h c and v_h = W_uv,h c the two forms agree: the absorbed
 * query is [W_uk,h^T q_nope | q_pe] and the head's output W_uv,h o.  Those
 * products are plain matrix products and stay with the caller.
 *
 * Arithmetic of the two attention forms: scores, maxima, sums, accumulators and
 * the parts of a split call are fp32.  The softmax weights are rounded to bf16
 * for the product with the values, the operands' type of the tensor cores, after
 * their sum has been taken; with the rounding of out itself (2^-8 each) a value
 * is off by at most about 2^-7 sum_j p_j |v_j|.  Measured against 64 bits on
 * standard normal data: relative RMS 0.0017 to 0.0023, of which 0.0017 are the
 * rounding of out.  lse is fp32 and does not see the weights' rounding.
 *
 * Conventions are those of kda.h: caller-owned device memory, 16-byte aligned
 * tensor pointers, work enqueued on the given stream, argument errors returned
 * before any launch, inconsistent device values (lengths, page ids, slots)
 * found by the kernels and reported by kda_get_status(stream).  Nothing is
 * allocated and no pointer is kept; calls may be captured into CUDA graphs
 * once each has been used on the device.
 */
#ifndef KDA_LATENT_H_
#define KDA_LATENT_H_

#include "kda.h"

#ifdef __cplusplus
extern "C" {
#endif

#define KDA_LATENT_DIM 512     /* latent values of a cache row (also the value width) */
#define KDA_LATENT_PE_DIM 64   /* shared key values of a cache row */
#define KDA_LATENT_ROW 576     /* a cache row, and a head of the absorbed query */
#define KDA_LATENT_QK_DIM 192  /* a head of the expanded query: 128 own + 64 shared */
#define KDA_LATENT_V_DIM 128   /* a head of the expanded values */

/* ---- further status codes ---- */
#define KDA_ERR_STRIDE 15      /* a stride is not a multiple of 16 bytes or rows overlap */
#define KDA_ERR_SCALE 16       /* scale is not a positive finite number */
#define KDA_ERR_PAGE_SIZE 17   /* page_size is not a positive multiple of 8 */
#define KDA_ERR_BAD_LENGTHS 18 /* (device status) a length is negative, or longer than its table, slots or pages allow */
#define KDA_ERR_NO_PAGES 19    /* (device status) kda_latent_plan: too few free pages */
#define KDA_ERR_BAD_PAGE 20    /* (device status) a page id or slot outside the cache */

/*
 * Block tables and slot maps from request lengths.  Request b holds
 * cached_lens[b] tokens in the pages block_table[b][0 .. ceil(cached / page_size))
 * and gets new_lens[b] tokens.  The pages it lacks are taken from free_pages in
 * order (requests in order, a request's pages in order) and written into its row
 * of the table; entries behind a request's last page are left as they are.
 *
 *  cached_lens, new_lens : int32 [B]
 *  block_table : int32 [B, max_pages], rows table_stride entries apart; read and written
 *  free_pages  : int32 [num_free]
 *  seq_lens    : int32 [B], out: cached + new
 *  cu_seqlens  : int64 [B + 1], out: offsets of the requests' new tokens, packed
 *  slot_map    : int64 [T], out: cache slot (page * page_size + offset) of every
 *                packed new token; -1 behind the last one (T is a capacity)
 *  pages_taken : int32 [1], out: entries of free_pages used (always the first ones)
 * If the lengths do not fit (a negative one, more than T new tokens, a request
 * beyond max_pages pages or 2^31 - 1 tokens: KDA_ERR_BAD_LENGTHS) or free_pages
 * is too short (KDA_ERR_NO_PAGES), the status word is set and nothing is
 * planned: the table stays, seq_lens = cached_lens, cu_seqlens 0, slot_map -1,
 * pages_taken 0.  B is at most 16384.
 */
typedef struct kda_latent_plan_args {
  const int32_t *cached_lens, *new_lens;
  int32_t *block_table;
  int64_t table_stride;
  const int32_t *free_pages;
  int32_t *seq_lens;
  int64_t *cu_seqlens;
  int64_t *slot_map;
  int32_t *pages_taken;
  int64_t B, max_pages, num_free, page_size, T;
} kda_latent_plan_args;

int kda_latent_plan(const kda_latent_plan_args *args, void *stream);

/* The paged cache: bf16 rows of 576 values; row (page p, offset i) starts at
 * data + p * page_stride + i * token_stride (elements, multiples of 8).
 * page_size is a multiple of 8. */
typedef struct kda_latent_cache {
  void *data;
  int64_t num_pages, page_size, page_stride, token_stride;
} kda_latent_cache;

/*
 * New tokens' rows into the cache: row slot_map[t] = [y_t | k_pe_t] with
 *   y_t = c_t / sqrt(mean(c_t^2) + eps) * norm_weight     (fp32, rounded once)
 * or y_t = c_t where norm_weight is NULL.
 *
 *  c         : bf16 [T, 512], rows c_stride elements apart (multiple of 8)
 *  k_pe      : bf16 [T, 64],  rows k_pe_stride elements apart (multiple of 8)
 *  slot_map  : int64 [T]; a negative slot skips its token, one past the cache
 *              skips it and sets KDA_ERR_BAD_PAGE.  Slots should be distinct.
 *  norm_weight : fp32 [512] or NULL
 */
typedef struct kda_latent_append_args {
  const void *c, *k_pe;
  int64_t c_stride, k_pe_stride;
  const int64_t *slot_map;
  kda_latent_cache cache;
  const float *norm_weight;
  float eps;
  int64_t T;
} kda_latent_append_args;

int kda_latent_append(const kda_latent_append_args *args, void *stream);

/*
 * Absorbed attention of the newest R tokens of every request over the paged
 * cache (which already holds them).  Token i of request b sees the rows
 * j < seq_lens[b] - (R - 1 - i); a token that sees none gives zeros and -inf.
 *
 *  q   : bf16 [B, R, H, 576], dense      out : bf16 [B, R, H, 512], dense
 *  lse : fp32 [B, R, H] or NULL: natural log of the sum of exp(s)
 *  block_table : int32 [B, max_pages], rows table_stride entries apart
 *  seq_lens    : int32 [B], read on the device only.  A length outside
 *                [0, max_pages * page_size] is taken as the nearer bound and
 *                sets KDA_ERR_BAD_LENGTHS; a page id outside the cache reads as
 *                zero rows and sets KDA_ERR_BAD_PAGE.
 * What the cache holds behind a request's length is never used, whatever it is;
 * the rows within it have to be finite (with R > 1 also for the tokens that do not
 * see the last of them: they take part with weight 0).
 * Results do not depend on anything but the arguments (fixed order of sums).
 */
typedef struct kda_latent_decode_args {
  const void *q;
  kda_latent_cache cache;
  const int32_t *block_table;
  int64_t table_stride, max_pages;
  const int32_t *seq_lens;
  float scale;
  void *out;
  float *lse;
  int64_t B, R, H;
} kda_latent_decode_args;

/* Device scratch of kda_latent_decode on the current device (0 for arguments it
 * would reject); garbage afterwards, needs no initialisation, 256-byte aligned. */
size_t kda_latent_decode_workspace_bytes(const kda_latent_decode_args *args);
int kda_latent_decode(const kda_latent_decode_args *args, void *workspace, size_t workspace_bytes,
                      void *stream);

/*
 * Expanded attention of prompts.  Sequence n has queries i < Lq and keys
 * j < Lk (Lk may exceed Lq: context that is already there); query i sees every
 * key, or with KDA_LATENT_CAUSAL those with j <= i + Lk - Lq.  A query that
 * sees none gives zeros and -inf.
 *
 *  q    : bf16 [B, Tq, H, 192]  token / head strides q_stride_t / q_stride_h
 *  k    : bf16 [B, Tk, H, 128]  k_stride_t / k_stride_h   (the heads' own key channels)
 *  k_pe : bf16 [B, Tk, 64]      k_pe_stride_t             (shared by the heads)
 *  v    : bf16 [B, Tk, H, 128]  v_stride_t / v_stride_h
 *         strides in elements, multiples of 8; batch row b starts at token b * T,
 *         so k and v may be views of one up-projection's [.., H, 256] output
 *  out  : bf16 [B, Tq, H, 128], dense      lse : fp32 [B, Tq, H] or NULL
 *  cu_seqlens_q, cu_seqlens_k : int64 [N + 1] (B == 1, packed) or both NULL
 *         (N == B, sequence n = batch row n).  Checked on the device as in kda.h;
 *         a violation of either sets KDA_ERR_BAD_SEQLENS and nothing is written.
 *         (N == 0 with Tq or Tk > 0 is refused with KDA_ERR_BAD_SEQLENS at once.)
 * Rows of other sequences (and past the tensors) never touch a result; within a
 * sequence, keys and values have to be finite (behind the causal edge too, as there).
 *
 * workspace: kda_latent_prefill_workspace_bytes bytes, aligned to 256.  A call with
 * few blocks of queries and many keys has its keys split over the SMs and the parts
 * joined, for which it needs some; a dense call with workspace NULL is not split.
 */
#define KDA_LATENT_CAUSAL 0x1u
#define KDA_LATENT_SPLIT_KEYS 4096 /* dense calls with fewer keys are never split and need no workspace */
typedef struct kda_latent_prefill_args {
  const void *q, *k, *k_pe, *v;
  int64_t q_stride_t, q_stride_h, k_stride_t, k_stride_h, k_pe_stride_t, v_stride_t, v_stride_h;
  float scale;
  void *out;
  float *lse;
  const int64_t *cu_seqlens_q, *cu_seqlens_k;
  int64_t B, Tq, Tk, H, N;
  uint32_t flags;
} kda_latent_prefill_args;

size_t kda_latent_prefill_workspace_bytes(const kda_latent_prefill_args *args);
int kda_latent_prefill(const kda_latent_prefill_args *args, void *workspace, size_t workspace_bytes,
                       void *stream);

#ifdef __cplusplus
}
#endif

#endif /* KDA_LATENT_H_ */
