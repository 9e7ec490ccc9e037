/*
 * dspark_kv4.h -- a paged key/value cache held in 4 bits, for the target
 * model's side of speculative decoding: storing (with rotary positions) and
 * reading rows, attention of a step's rows over the cache or over the pages of it
 * that a cheap score selects, and the bookkeeping of its pages (the same library
 * as dspark_markov.h; its error codes and conventions apply).
 *
 * A step of a serving loop: dspark_pages_grow makes room for the P + 1 rows of
 * a verification, dspark_kv4_append stores their keys and values
 * (dspark_kv4_append_rotated turns them by their positions first),
 * dspark_kv4_attention attends (or, over long contexts, dspark_kv4_bound_pages,
 * dspark_kv4_select and dspark_kv4_attention_selected), dspark_greedy_accept (or the probabilistic
 * form) decides, and dspark_pages_trim cuts the requests back to the accepted
 * length.  A slot to which dspark_pages_grow grants nothing keeps its length: in
 * that step its request gets no rows, or slot -1, or they are stored over its
 * last tokens.  dspark_pages_fork starts branches that share their pages.  All
 * lengths, page tables and reference counts live on the device: no entry
 * point synchronises the host or allocates, and all are safe to capture in a
 * CUDA graph.
 */
#ifndef DSPARK_KV4_H
#define DSPARK_KV4_H

#include "dspark_markov.h"

#ifdef __cplusplus
extern "C" {
#endif

/* ---- element types ------------------------------------------------------ */
#define DSPARK_DTYPE_BF16 0
#define DSPARK_DTYPE_F16 1
#define DSPARK_DTYPE_F32 2 /* dspark_kv4_read only */

#define DSPARK_KV4_MAX_BATCH 4096    /* requests of one call */
#define DSPARK_PAGES_MAX_SLOTS 4096  /* slots of one dspark_pages_* call */

/*
 * One layer's cache.  A page holds `page_size` tokens; page p starts at byte
 * p * page_stride of `data` and holds one record for each key/value head, one
 * after the other, of page_size * (head_dim + head_dim / 8) bytes:
 *   key codes   [page_size][head_dim / 2]    byte j: element 2j in the low
 *   value codes [page_size][head_dim / 2]    four bits, 2j + 1 in the high
 *   key scales  [page_size][head_dim / 16]   one byte for 16 elements
 *   value scales[page_size][head_dim / 16]
 * A code is E2M1 (sign, then 0, .5, 1, 1.5, 2, 3, 4, 6), a scale E4M3, and an
 * element stands for RN(code * scale * g) with the head's FP32 scale g
 * (code * scale is exact; a scale byte that is an E4M3 NaN, which
 * dspark_kv4_append never writes, reads as 448).  So every byte pattern reads
 * as a finite number.
 *   data: device, 16-byte aligned; page_stride in bytes, a multiple of 16.
 *   page_size 16, 32, 64, 128 or 256; head_dim 64 or 128; kv_heads >= 1.
 *   k_scale, v_scale: device [kv_heads] FP32 (finite, not 0), or NULL for 1.
 */
typedef struct dspark_kv4_cache {
  void *data;
  int64_t page_stride;
  int32_t num_pages;
  int32_t page_size;
  int32_t kv_heads;
  int32_t head_dim;
  const float *k_scale;
  const float *v_scale;
} dspark_kv4_cache;

/*
 * The requests of a step.  Request i is in cache slot slots[i] (i itself when
 * slots is NULL) and has the rows row_start[i] .. row_start[i + 1] - 1 of the
 * step's tensors: the last rows of the lens[slot] tokens its cache holds, so
 * its row j is at position lens[slot] - n + j (n its number of rows; a row at
 * a negative position stores, reads and sees nothing).  Token t of a slot is
 * in row t % page_size of page table[slot * table_stride + t / page_size].
 *   row_start [batch + 1], lens [max_slots], table [max_slots][table_stride]:
 *   device int32.  A request may have no rows.  0 <= batch <=
 *   DSPARK_KV4_MAX_BATCH; max_pages <= table_stride columns are used.
 *   total_rows: rows of the tensors; max_rows: the most rows of one request.
 *   These and batch and max_pages choose the attention's kernel and the size of
 *   its workspace (lengths are on the device): tables much wider than the
 *   requests are long may get a slower one.  A request with more rows than
 *   max_rows is still computed.  A call of 2^31 - 256 or more blocks of 64 tokens
 *   (each tile of 8 to 256 rows of a request and key/value head with each block
 *   that it sees, and 7 more; larger tiles are taken where the tables allow so
 *   many) is not: its rows are NaN.
 * Lengths are taken as at most max_pages * page_size and 2^31 - 4097, row
 * numbers as within [0, total_rows]; a slot outside [0, max_slots) holds no
 * tokens, and tokens whose page id is outside [0, num_pages) are not there: they
 * are not stored, read as 0 and are not attended to.  Two requests of a call may
 * share pages, as long as no call stores to a page that two of them hold.
 */
typedef struct dspark_kv4_batch {
  int32_t batch;
  int32_t total_rows;
  int32_t max_rows;
  int32_t max_pages;
  int32_t max_slots;
  int32_t reserved; /* 0 */
  const int32_t *row_start;
  const int32_t *slots;
  const int32_t *lens;
  const int32_t *table;
  int64_t table_stride;
} dspark_kv4_batch;

/*
 * dspark_kv4_append -- quantise and store the keys and values of the rows.
 *   k, v: device [total_rows][kv_heads][head_dim] of `dtype` (BF16 or F16),
 *   element strides (k_row, k_head, 1); 16-byte loads where pointers and
 *   strides allow, else 2-byte loads (2-byte alignment is needed).
 * For each 16 elements: y = RN(x / g) (NaN as 0), the scale is
 * E4M3(min(RN(max|y| / 6), 448)) to nearest even, and the codes are
 * E2M1(RN(y / scale)), nearest even, saturating (all 0 where the scale is 0).
 * One kernel on `stream`.
 */
DSPARK_API int dspark_kv4_append(const dspark_kv4_cache *cache, const dspark_kv4_batch *batch, const void *k,
                                 int64_t k_row, int64_t k_head, const void *v, int64_t v_row, int64_t v_head,
                                 int32_t dtype, cudaStream_t stream);

/*
 * dspark_kv4_read -- the cached rows as the numbers they stand for, rounded
 * once more to `dtype` (BF16, F16 or F32).  Shapes and strides as for
 * dspark_kv4_append; k or v may be NULL to read one of the two.  A request
 * whose rows are as many as its tokens is read whole.  One kernel.
 */
DSPARK_API int dspark_kv4_read(const dspark_kv4_cache *cache, const dspark_kv4_batch *batch, void *k, int64_t k_row,
                               int64_t k_head, void *v, int64_t v_row, int64_t v_head, int32_t dtype,
                               cudaStream_t stream);

/*
 * dspark_kv4_attention -- softmax attention of the rows over their requests'
 * caches.  Query head h reads key/value head h / (q_heads / kv_heads).  A row
 * at position p sees tokens 0 .. p, with window > 0 the last `window` of them
 * (p - window + 1 .. p).
 *   s_t = scale * sum_d q_d k_td,  out = sum_t exp(s_t) v_t / sum_t exp(s_t),
 *   lse = log sum_t exp(s_t);  a row that sees nothing gets out 0, lse -inf.
 *   Scores are taken to lie below 2^23 in magnitude, where FP32 still holds
 *   whole numbers and halves: a row with larger ones may be 0 or NaN.
 *   q, out: device [total_rows][q_heads][head_dim] of `dtype` (BF16 or F16),
 *   element strides (row, head, 1); 2-byte alignment is needed, 16-byte loads
 *   and stores where pointers and strides allow.  out must not overlap q.
 *   lse: device [total_rows][q_heads] FP32, or NULL.
 *   scale: finite.  q_heads a multiple of kv_heads.  window >= 0 (0: none).
 *   workspace: device, 256-byte aligned, at least
 *   dspark_kv4_attention_workspace_bytes bytes; its contents on entry do not
 *   matter, and it belongs to the call until its kernels have run.
 * Products of queries and cached keys and values are taken on tensor cores
 * with FP16 operands (BF16 queries enter as FP16 of q 2^e per row: exact for
 * every element within 2^-28 of the row's largest), with FP32 accumulation;
 * weights enter the second product as FP16 (with F16 results as the sum of two
 * FP16 numbers), maxima and sums are FP32.  Rows
 * of requests that are not in the batch are left unwritten.  Two kernels on
 * `stream`; deterministic.  A bounded device wait that gave up (never in
 * correct operation) leaves NaN in the rows concerned.
 */
typedef struct dspark_kv4_attention_args {
  const void *q;
  int64_t q_row, q_head;
  void *out;
  int64_t out_row, out_head;
  float *lse;
  int32_t q_heads;
  int32_t dtype;
  float scale;
  int32_t window;
  void *workspace;
  size_t workspace_bytes;
} dspark_kv4_attention_args;

DSPARK_API size_t dspark_kv4_attention_workspace_bytes(const dspark_kv4_cache *cache, const dspark_kv4_batch *batch,
                                                       int32_t q_heads);
DSPARK_API int dspark_kv4_attention(const dspark_kv4_cache *cache, const dspark_kv4_batch *batch,
                                    const dspark_kv4_attention_args *args, cudaStream_t stream);

/*
 * dspark_kv4_append_rotated -- dspark_kv4_append with rotary positions on the
 * way: the rows' keys are rotated before they are quantised, their queries
 * rotated and rounded once to `dtype`.
 *   The first `dims` elements of a head (a multiple of 32, at least 32, at most
 *   head_dim) are turned in pairs (a, b): elements i and i + dims / 2, or with
 *   `interleaved` not 0 elements 2 i and 2 i + 1, for i below dims / 2:
 *     a' = RN(RN(a c) - RN(b s)),  b' = RN(RN(b c) + RN(a s))  in FP32,
 *   c = cos[p * stride + i], s = sin[p * stride + i] for the row's position p;
 *   the others stay.  cos, sin: device FP32, [positions][dims / 2], stride >=
 *   dims / 2 elements from row to row, 4-byte aligned (16-byte loads where
 *   pointers and stride allow); any scaling of the angles is in them.
 *   at: device int32 [total_rows], each row's p; NULL for its position in the
 *   cache.  A row whose p is outside [0, positions) stores nothing and its
 *   rotated queries are NaN; one at a negative position in the cache stores
 *   nothing and its queries become 0.
 *   k, v as for dspark_kv4_append.  q, q_out: device [total_rows][q_heads]
 *   [head_dim] of `dtype`, element strides (row, head, 1); q_out may be q with
 *   q's strides, else they must not overlap.  q NULL (and q_out NULL): keys and
 *   values only.  q_heads >= 1, any number with 2 * kv_heads + q_heads < 2^31 -
 *   1024.  Rows of q_out of no request are left unwritten.  One kernel on `stream`.
 */
typedef struct dspark_kv4_rotation {
  const float *cos, *sin;
  int64_t stride;
  int32_t positions;
  int32_t dims;
  int32_t interleaved;
  int32_t reserved; /* 0 */
  const int32_t *at;
} dspark_kv4_rotation;

typedef struct dspark_kv4_rotated_args {
  const void *k;
  int64_t k_row, k_head;
  const void *v;
  int64_t v_row, v_head;
  const void *q;
  int64_t q_row, q_head;
  void *q_out;
  int64_t out_row, out_head;
  int32_t q_heads;
  int32_t dtype;
} dspark_kv4_rotated_args;

DSPARK_API int dspark_kv4_append_rotated(const dspark_kv4_cache *cache, const dspark_kv4_batch *batch,
                                         const dspark_kv4_rotation *rotation, const dspark_kv4_rotated_args *args,
                                         cudaStream_t stream);

/*
 * Attention over a few pages of a long cache that a cheap score selects for
 * each row and key/value head: dspark_kv4_bound_pages after each append,
 * dspark_kv4_select, dspark_kv4_attention_selected.
 *
 * dspark_kv4_bound_pages -- brings the bounds of the pages that hold the
 * batch's rows up to date, over all of a page's tokens below its slot's length.
 *   Page p's bounds start at byte p * bounds_stride and hold for each head
 *   2 * head_dim + 16 bytes: lo [head_dim] and hi [head_dim], int8, then m, FP32,
 *   then 12 bytes of 0.  With x = code * scale (exact; without the head's FP32
 *   scale) of the page's keys, m is the largest |x|, and an element of lo (of hi)
 *   the nearest whole number, ties to even, of RN(127 x / m) for the smallest
 *   (largest) x of its dimension; all 0 where m is 0.  A scale byte that is NaN
 *   counts as 448, as everywhere: m is finite.
 *   bounds: device, 16-byte aligned; bounds_stride in bytes, a multiple of 16, at
 *   least kv_heads * (2 * head_dim + 16).
 * A slot that is cut back (dspark_pages_trim) needs no call: its last page is
 * done again when rows are stored to it.  Pages that dspark_pages_compact moves
 * have their bounds moved by dspark_pages_copy; a shared last page that
 * dspark_pages_grow has copied needs them only if the slot gets no rows.  One
 * kernel on `stream`.
 */
DSPARK_API int dspark_kv4_bound_pages(const dspark_kv4_cache *cache, const dspark_kv4_batch *batch, void *bounds,
                                      int64_t bounds_stride, cudaStream_t stream);

/*
 * The pages that rows attend to.  pages: device int32 [rows][kv_heads][top],
 * contiguous: page ids in the order of their tokens, -1 behind the last.  lens:
 * device int32 [rows]: the tokens of a row's pages, all pages whole but the last;
 * the same for all of its heads; 0: the row sees nothing, -1: there is no such
 * row.  top >= 1.
 */
typedef struct dspark_kv4_selection {
  int32_t *pages;
  int32_t *lens;
  int32_t rows;
  int32_t top;
} dspark_kv4_selection;

/*
 * dspark_kv4_select -- writes the selection of the batch's rows (selection->rows
 * = total_rows).  A row at position p has n = p / page_size + 1 pages; if n <= top
 * it gets all of them, else for each head the first `first`, the last `last` and,
 * to make `top`, those of the largest scores, ties to the lower page:
 *   a_d = sum of min(q_d, 0), b_d = sum of max(q_d, 0) over the queries q of the
 *   head's group, in their order, in FP32 (NaN as 0, magnitudes held to 2^100; -q
 *   for q where the head's key scale is negative); as int8, with t the largest
 *   |a_d|, |b_d|: the nearest whole numbers, ties to even, of RN(RN(127 a_d) / t)
 *   (all 0 where t is 0);
 *   score = RN(m * sum_d (a_d lo_d + b_d hi_d)), the sum exact:
 *   about the sum, over the group's queries, of the largest product that each could
 *   have with a key within the page's bounds.  (One key need not reach all of them,
 *   and eight bits round either way, a page's sum by up to m / 254 times that of all
 *   |a_d|, |b_d| and t / 254 times that of all its keys' least and largest |x|.)
 *   A page whose id is outside [0, num_pages) comes behind all others; a NaN (of an m
 *   that dspark_kv4_bound_pages did not write: its own are finite) counts as the
 *   largest.
 * The lists hold page ids; where they are equal to the table's, in its order.
 *   q: device [total_rows][q_heads][head_dim] of `dtype` (BF16 or F16), element
 *   strides (row, head, 1), 2-byte alignment, 16-byte loads where they allow.
 *   q_heads a multiple of kv_heads, at most 2^30; total_rows * q_heads below 2^31.
 *   first >= 0, last >= 1, first + last <= top.
 *   workspace: device, 256-byte aligned, at least dspark_kv4_select_workspace_bytes
 *   bytes (for each row and head 2 head_dim and 4 max_pages, to a multiple of 16,
 *   and 256; 256 alone where max_pages <= top); it belongs to the call until its
 *   kernels have run, and may then be the attention's.
 * Rows of no request get lens -1.  One kernel on `stream`, or three; which, goes by
 * total_rows, batch, kv_heads and max_pages (lengths are on the device): tables much
 * wider than the requests are long may get the slower one, with the same lists.
 */
typedef struct dspark_kv4_select_args {
  const void *q;
  int64_t q_row, q_head;
  int32_t q_heads;
  int32_t dtype;
  int32_t first;
  int32_t last;
  void *workspace;
  size_t workspace_bytes;
} dspark_kv4_select_args;

DSPARK_API size_t dspark_kv4_select_workspace_bytes(const dspark_kv4_cache *cache, const dspark_kv4_batch *batch,
                                                    const dspark_kv4_selection *selection);
DSPARK_API int dspark_kv4_select(const dspark_kv4_cache *cache, const dspark_kv4_batch *batch, const void *bounds,
                                 int64_t bounds_stride, const dspark_kv4_selection *selection,
                                 const dspark_kv4_select_args *args, cudaStream_t stream);

/*
 * dspark_kv4_attention_selected -- dspark_kv4_attention of each row over its
 * heads' pages (arguments, arithmetic and limits as there, so that with BF16 results
 * a weight is one FP16 number in the second product, with F16 results two; window
 * must be 0, and q, out and lse have selection->rows rows).  Rows of lens -1 are left
 * unwritten.
 * A pair of kernels on `stream` for each 4096 rows; deterministic.
 */
DSPARK_API size_t dspark_kv4_attention_selected_workspace_bytes(const dspark_kv4_cache *cache,
                                                                const dspark_kv4_selection *selection,
                                                                int32_t q_heads);
DSPARK_API int dspark_kv4_attention_selected(const dspark_kv4_cache *cache, const dspark_kv4_selection *selection,
                                             const dspark_kv4_attention_args *args, cudaStream_t stream);

/*
 * The pages of a cache (of every layer that shares its page tables).
 *   refs  [num_pages]: how many slots hold a page; 0 is a free page.
 *   table [max_slots][table_stride]: a slot's page ids in order; the entries
 *         behind its last page are not read.
 *   lens  [max_slots]: a slot's tokens; it holds ceil(len / page_size) pages.
 * All device int32, owned by the caller; a new pool is refs = 0, lens = 0.
 * A call takes up to DSPARK_PAGES_MAX_SLOTS slots, which must differ from one
 * another (for a fork: the destinations, from the sources too); a slot outside
 * [0, max_slots) is skipped.  n >= 0.  Calls on one pool are to be ordered
 * (one stream, or events).  One kernel each, unless said otherwise.
 */
typedef struct dspark_page_pool {
  int32_t num_pages;
  int32_t page_size; /* >= 1 */
  int32_t max_slots;
  int32_t max_pages; /* <= table_stride: the most pages of a slot */
  int32_t *refs;
  int32_t *table;
  int64_t table_stride;
  int32_t *lens;
} dspark_page_pool;

/* dspark_pages_trim -- cuts slot slots[i] back to new_len[i] tokens (0 frees
 * it): pages behind ceil(new_len / page_size) lose a reference, and their
 * table entries become -1.  A new_len below 0 or not below the slot's length
 * leaves it as it is. */
DSPARK_API int dspark_pages_trim(const dspark_page_pool *pool, int32_t n, const int32_t *slots,
                                 const int32_t *new_len, cudaStream_t stream);

/* dspark_pages_fork -- slot dst[i] becomes a branch of slot src[i]: the same
 * tokens on the same pages, which gain a reference each.  What dst[i] held
 * before loses its references; its table entries behind the branch become -1
 * up to the last page it held.  Several branches of one source may be made in
 * a call.  A pair with either slot outside [0, max_slots) is skipped. */
DSPARK_API int dspark_pages_fork(const dspark_page_pool *pool, int32_t n, const int32_t *src, const int32_t *dst,
                                 cudaStream_t stream);

/* dspark_pages_grow -- makes room for add[i] >= 0 more tokens in slot
 * slots[i] and adds them to its length.  New pages are the lowest free ones,
 * given out in the order of the list and, in a slot, of its pages.  Where the
 * slot's last page is partly filled and held by others too, the slot first
 * gets a page of its own for it and (copy_src[i], copy_dst[i]) = (old page, new
 * page) asks for the data to be copied (dspark_pages_copy, for every layer);
 * else the pair is (-1, -1).  If all holders of that page are in the list,
 * each with add > 0 and within max_pages, the last of them keeps it: it needs
 * no copy, as the others leave the page in this call.  granted[i] = 1, or 0
 * where the slot is left as it was: the free pages did not reach it (the sum of
 * the pages wanted by it and the slots listed before it, granted or not, is
 * more than were free at the call), it would exceed max_pages, add[i] < 0, or
 * the page that it would keep is still held by a slot that was refused.  After
 * the call no other slot holds the page that a granted slot writes to next.  A
 * page that the call gives up is free for the next call. */
DSPARK_API int dspark_pages_grow(const dspark_page_pool *pool, int32_t n, const int32_t *slots, const int32_t *add,
                                 int32_t *copy_src, int32_t *copy_dst, int32_t *granted, cudaStream_t stream);

/* dspark_pages_compact -- moves the pool's L live pages to ids 0 .. L - 1: the
 * k-th live page from id L on moves to the k-th free id below L.  Writes
 * map [num_pages] (each live page's new id, -1 for a free one), the moves
 * move_src, move_dst [num_pages] (count[0] of them, in order; -1 behind), and
 * the pool's table and refs after the move to table_out [max_slots] with
 * table_stride, and refs_out [num_pages] (entries below 0 or behind num_pages
 * stay as they are).  The pool itself is only read, so a step in flight may
 * still use it: moved data go to pages that were free.  table_out == table and
 * refs_out == refs work in place.  Then copy the data with
 * dspark_pages_copy and that count for every layer.  Two kernels. */
DSPARK_API int dspark_pages_compact(const dspark_page_pool *pool, int32_t *table_out, int32_t *refs_out,
                                    int32_t *map, int32_t *move_src, int32_t *move_dst, int32_t *count,
                                    cudaStream_t stream);

/* dspark_pages_copy -- copies page src[i] to page dst[i] in each of `layers`
 * layers: page p of layer l is the page_bytes bytes at data + l *
 * layer_stride + p * page_stride (bytes; all multiples of 16, data 16-byte
 * aligned).  Pairs with a negative or too large id are skipped.  count: device
 * int32 or NULL; with it only the first min(n, count[0]) pairs are copied.  No
 * page may be a destination and also a source, or twice a destination.
 * n >= 0. */
DSPARK_API int dspark_pages_copy(void *data, int32_t num_pages, int64_t page_bytes, int64_t page_stride,
                                 int32_t layers, int64_t layer_stride, int32_t n, const int32_t *src,
                                 const int32_t *dst, const int32_t *count, cudaStream_t stream);

#ifdef __cplusplus
}
#endif
#endif /* DSPARK_KV4_H */
