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
 * Beside them: kda_latent_decode_shared, the absorbed form for requests that share
 * long prefixes, and calls for the pages that several requests hold
 * (kda_latent_fork, _release, _compact, _copy).
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
#define KDA_ERR_BAD_LENGTHS 18 /* (device status) a length is negative, or longer than its table, slots or pages allow;
                                  or would grow in a page that others hold; or a request's number does not fit */
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
 *  shares      : int32 [num_pages] or NULL: the holders of the cache's pages beyond the
 *                first (see the calls on pages below).  Where given, a request with new
 *                tokens whose last page is not whole has to be its only holder: a row that
 *                kda_latent_release cut within a page of others does not write into theirs
 * If the lengths do not fit (a negative one, more than T new tokens, a request
 * beyond max_pages pages or 2^31 - 1 tokens, new tokens for a page that others hold:
 * KDA_ERR_BAD_LENGTHS) or free_pages
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
  const int32_t *shares;
  int64_t num_pages;             /* entries of shares */
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
 * Absorbed attention of a batch whose requests share long prefixes: the result of
 * kda_latent_decode on the same arguments, with each shared prefix read once for
 * all requests of its group instead of once a request.
 *
 *  decode      : the arguments of kda_latent_decode; requests of a group are
 *                neighbours, and each request's row of the table names its whole
 *                context, prefix first (as kda_latent_fork leaves it)
 *  cu_groups   : int64 [G + 1]: group g has the requests [cu_groups[g], cu_groups[g + 1])
 *  prefix_lens : int32 [G]: the first prefix_lens[g] tokens hold the same values for
 *                all requests of the group.  Where only whole pages are the same
 *                pages, the rows behind them may be copies
 * Which request's row names the pages that are read for a shared prefix is not
 * said.  A request that does not see the whole prefix (a shorter or an empty one)
 * is taken on its own, as are the requests of groups of one.  The prefix_lens of a
 * group without requests is not looked at; another below 0 or beyond the table is
 * taken as the nearer bound and sets KDA_ERR_BAD_LENGTHS; offsets that do not go from 0
 * to B without decreasing set KDA_ERR_BAD_SEQLENS, and every request is taken on its
 * own.  B * R * H is below 2^31 - 128, a table
 * holds at most 2^30 tokens, and G is at most KDA_LATENT_SHARED_GROUPS.
 * Cached rows that are not finite touch no result of a request that does not see them
 * (such a call is slow: a request's tokens take part with weight 0 in the products of its
 * group's others, and what that spoils is computed anew).  A request's own rows have to be
 * finite as in kda_latent_decode: whether one that is not reaches the new tokens before it
 * depends on the form that a call takes.
 * What the cache holds behind a request's length is never used, whatever it is.
 * Parts are joined in fp32, so outputs have the error of kda_latent_decode's; they are
 * not bit for bit the same, but do not depend on anything but the arguments.
 * Where the tables hold little (B * max_pages * page_size tokens times R H, or 16 if that
 * is more, are at most KDA_LATENT_SHARED_LEAST) and the rows are few (R H at most 32, or
 * B R H at most KDA_LATENT_SHARED_ROWS) the call is kda_latent_decode, which is faster
 * there; the values of cu_groups and prefix_lens are then not looked at.
 */
#define KDA_LATENT_SHARED_LEAST 2097152
#define KDA_LATENT_SHARED_ROWS 512
#define KDA_LATENT_SHARED_GROUPS 16384
typedef struct kda_latent_decode_shared_args {
  kda_latent_decode_args decode;
  const int64_t *cu_groups;
  const int32_t *prefix_lens;
  int64_t G;
} kda_latent_decode_shared_args;

/* As kda_latent_decode_workspace_bytes. */
size_t kda_latent_decode_shared_workspace_bytes(const kda_latent_decode_shared_args *args);
int kda_latent_decode_shared(const kda_latent_decode_shared_args *args, void *workspace, size_t workspace_bytes,
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

/* ---- pages that several requests hold ----
 *
 * Requests that share a prefix (samples or beams of one prompt, a common system
 * prompt) hold the same pages.  shares[page] (int32, one a page of the cache)
 * counts a page's holders beyond the first: 0 where one row of the table holds
 * it, so the pages that kda_latent_plan takes are right with zeros, and whole
 * pages are never written again.  A request holds the pages
 * block_table[b][0 .. ceil(cached_lens[b] / page_size)); B is at most 16384.
 * Every list of pages is in an order of its own, not of time.
 */

/*
 * Requests that go on from others: child f = children[f] gets the first
 * fork_lens[f] tokens of request parents[f] (all of them where fork_lens is
 * NULL).  Whole pages are shared: their ids go into the child's row, their counts
 * up by one.  The rows of a last page that is not whole are copied into the next
 * page of free_pages (children in order).  Entries behind a child's last page are
 * left as they are; what a child's row held before has to be released first (its
 * cached length is then 0).
 *
 *  parents, children, fork_lens : int32 [F].  No child twice, and none that is a
 *                parent in the same call; one parent may have many children
 *  block_table : int32 [B, max_pages]; the children's rows are written
 *  free_pages  : int32 [num_free]
 *  shares      : int32 [num_pages], read and written
 *  seq_lens    : int32 [B], out (another buffer than cached_lens): the children's
 *                tokens, else cached_lens
 *  pages_taken : int32 [1], out: entries of free_pages used (always the first ones)
 * Numbers of requests outside [0, B), lengths that do not fit, a child twice, as parent
 * or with tokens set KDA_ERR_BAD_LENGTHS, too short a free_pages KDA_ERR_NO_PAGES, and
 * nothing is forked (seq_lens = cached_lens, pages_taken 0).  A page id outside the
 * cache sets KDA_ERR_BAD_PAGE; it is entered, but not counted or copied.
 */
typedef struct kda_latent_fork_args {
  const int32_t *parents, *children, *fork_lens, *cached_lens;
  int32_t *block_table;
  int64_t table_stride;
  const int32_t *free_pages;
  int32_t *shares;
  kda_latent_cache cache;
  int32_t *seq_lens, *pages_taken;
  int64_t F, B, max_pages, num_free;
} kda_latent_fork_args;

int kda_latent_fork(const kda_latent_fork_args *args, void *stream);

/*
 * Requests that give pages back: rows[f] keeps its first keep_lens[f] tokens (none
 * where keep_lens is NULL) and drops the pages behind them.  The count of a dropped
 * page goes down by one; pages whose last holder dropped them are listed.
 * A row that keeps part of a page which others hold must not grow from there: its
 * next tokens would be written into their page (kda_latent_plan refuses it where it is
 * given shares).  kda_latent_fork with fork_lens goes on from any place, as it copies
 * that part; the row itself is then released.
 *
 *  rows, keep_lens : int32 [F]; no row twice
 *  block_table : int32 [B, max_pages], left as it is (a request's length says
 *                which entries hold)
 *  shares      : int32 [num_pages], not negative, read and written
 *  seq_lens    : int32 [B], out (another buffer than cached_lens): keep_lens for
 *                the rows, else cached_lens
 *  pages       : int32 [num_pages], out: the pages that are free now, ascending,
 *                and -1 behind them
 *  count       : int32 [1], out: how many these are
 * A row outside [0, B) or twice, a length that does not fit or keep_lens beyond it
 * set KDA_ERR_BAD_LENGTHS, and nothing is released (count 0).  A page id outside
 * the cache sets KDA_ERR_BAD_PAGE and is passed over.  A page that more rows drop
 * than its count says is listed once.
 */
typedef struct kda_latent_release_args {
  const int32_t *rows, *keep_lens, *cached_lens, *block_table;
  int64_t table_stride;
  int32_t *shares, *seq_lens, *pages, *count;
  int64_t F, B, max_pages, num_pages, page_size;
} kda_latent_release_args;

int kda_latent_release(const kda_latent_release_args *args, void *stream);

/*
 * Held pages together: with U pages held by the rows of the table, those with ids
 * from U on move to the ids below U that no row holds, both in ascending order, so
 * that pages U and behind are free.  Rows of pages are copied within the cache;
 * tables, counts and a map of old to new ids come out.
 *
 *  block_table, block_table_out : int32 [B, max_pages] (may be the same buffer, with
 *                the same stride); entries behind a request's last page are copied
 *  shares, shares_out : int32 [num_pages] (may be the same buffer); counts by new
 *                id, 0 from U on
 *  page_map    : int32 [num_pages], out: new id of every held page, -1 for others
 *  pages_used  : int32 [1], out: U
 * A length that does not fit sets KDA_ERR_BAD_LENGTHS and nothing moves: tables and
 * counts come out as they are, the map is the identity, pages_used num_pages.  A
 * page id outside the cache sets KDA_ERR_BAD_PAGE and comes out as it is.
 * num_pages is at most KDA_LATENT_COMPACT_PAGES.
 */
#define KDA_LATENT_COMPACT_PAGES 12582912
typedef struct kda_latent_compact_args {
  const int32_t *cached_lens, *block_table;
  int64_t table_stride;
  int32_t *block_table_out;
  int64_t table_out_stride;
  const int32_t *shares;
  int32_t *shares_out, *page_map, *pages_used;
  kda_latent_cache cache;
  int64_t B, max_pages;
} kda_latent_compact_args;

int kda_latent_compact(const kda_latent_compact_args *args, void *stream);

/*
 * Page src_pages[i] of one cache into page dst_pages[i] of another (or of the same
 * one, where no page is both read and written), with the same page_size; strides
 * may differ.  dst_pages should be distinct.  A page id outside its cache sets
 * KDA_ERR_BAD_PAGE and is passed over.
 *  src_pages, dst_pages : int32 [n]
 */
typedef struct kda_latent_copy_args {
  kda_latent_cache src, dst;
  const int32_t *src_pages, *dst_pages;
  int64_t n;
} kda_latent_copy_args;

int kda_latent_copy(const kda_latent_copy_args *args, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* KDA_LATENT_H_ */
