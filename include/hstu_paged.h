/*
 * hstu_paged.h — C ABI of libhstu_attn.so, second part: a paged K/V cache for the attention of
 * hstu_attn.h, the position rotation of Q and K, and the calls that fill and read the cache.
 *
 * A serving process keeps the K/V rows of its users' histories between requests (the reuse across
 * consecutive timestamps that hstu_attn_fwd_cached serves).  With one contiguous K/V matrix, a user
 * whose history grows moves everybody behind it; here the rows live in pages of a pool instead, and
 * a table names each user's pages:
 *
 *   hstu_rotary           position rotation of packed or strided Q and K (training), and its gradient
 *   hstu_paged_append     writes new K/V rows to the cache, rotating K (and Q) on the way
 *   hstu_paged_attn_fwd   attention of each user's new rows over its cached rows
 *
 * Status codes, the error word (hstu_attn_get_error), ownership, streams and threads are those of
 * hstu_attn.h.  All tensors are bf16 on the device, 16-byte aligned; products and sums are formed
 * in fp32, and outputs are rounded to bf16 once.  The attention rounds the weights silu(...) to bf16
 * as well, for their product with V, and takes their tanh from the hardware's approximation (within
 * 2^-10.9), as hstu_attn_fwd does.  The pages that hstu_attn.h cites give neither a cache layout
 * nor a rotation: these calls are additions of this library.
 *
 * Row strides.  A token tensor [rows, H, d] has its heads packed (element (t, h, c) at
 * t * ld + h * d + c) and rows `ld` elements apart, a multiple of 8 and at least H * d: a column
 * block of a wider projection can be passed as it is.
 *
 * New rows.  User b brings rows [q_offsets[b], q_offsets[b+1]) of the packed new-token tensors,
 * n_b of them; kv_len[b] is its length with them, so new row r is at position
 * kv_len[b] - n_b + r of its history.  n_b = 0 is legal, and so is a user with no earlier rows.
 * Inconsistent offsets or lengths (see each call) are reported as HSTU_ERR_BAD_OFFSETS and the user is
 * skipped; behind an offset that is smaller than the one before it, other users may be skipped too.
 * A call takes up to 2^30 users.
 */
#ifndef HSTU_PAGED_H_
#define HSTU_PAGED_H_

#include <stdint.h>

#include "hstu_attn.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * The cache.  Row `r` of page `p`, head h, column c of K is at
 * k[p * page_stride + r * row_stride + h * head_stride + c] (elements); V likewise.  So
 * [pages, page_size, H, d] and [pages, H, page_size, d] are both strides of the same form, and K and
 * V may be the two halves of one [pages, 2, ...] tensor.
 *   k, v          device, 16-byte aligned.
 *   strides       multiples of 8 elements, at least d.
 *   num_pages     pages of the pool (>= 1).
 *   page_size     rows of a page: a power of two, 8 .. 1024.
 *   page_table    device int32: user b's page i is page_table[b * table_ld + i].  Only entries
 *                 i < ceil(kv_len[b] / page_size) are read; the others may hold anything.  Users may
 *                 share pages that are only read (a common prefix).
 *   table_width   entries of a user that may be read; table_ld >= table_width.
 * Rows of a page past a user's last position are never used and may hold anything, NaN included.
 */
typedef struct hstu_paged_cache {
  void* k;
  void* v;
  int64_t page_stride, row_stride, head_stride;
  int32_t num_pages, page_size;
  const int32_t* page_table;
  int32_t table_width;
  int64_t table_ld;
} hstu_paged_cache_t;

/*
 * The rotation.  The first 2 * pairs columns of every head form pairs (x, y): columns (i, i + pairs),
 * or (2 i, 2 i + 1) if `interleaved`.  Pair i of the row at position(s) pos becomes
 *
 *     (x cos t - y sin t,  x sin t + y cos t),     t = pos[axis(i)] * freqs[i]   (radians)
 *
 * and the columns behind them pass unchanged.  With several axes (the place of an event in the
 * history, its time, ...) the pairs are shared out in runs: the first sections[0] pairs turn with
 * axis 0, the next sections[1] with axis 1, and so on.  Angles are reduced in 64 bits, so positions
 * may be Unix times: t is good to 1e-6 for |pos * freqs| up to 2^31 radians.
 *   freqs         device double [pairs], finite, 8-byte aligned.
 *   pairs         a multiple of 8, 2 * pairs <= d.
 *   axes          1 .. HSTU_MAX_AXES; sections[0 .. axes) are >= 0 and add up to `pairs`.
 *   positions     device int32: axis a of row t at positions[a * positions_ld + t].
 *                 hstu_paged_append accepts NULL with axes = 1: the row's place in the cache.
 */
#define HSTU_MAX_AXES 4

typedef struct hstu_rotation {
  const double* freqs;
  int32_t pairs, axes;
  int32_t sections[HSTU_MAX_AXES];
  int32_t interleaved;
  const int32_t* positions;
  int64_t positions_ld;
} hstu_rotation_t;

/*
 * hstu_rotary — rotates the rows of q and, unless k is NULL, of k.
 *   q, k          device bf16 [rows, H, d], rows q_ld / k_ld elements apart; d in {32, 64, 128}.
 *   inverse       0: as above.  1: by -t, which undoes the rotation and is also its gradient: the
 *                 rotation is orthogonal, so a gradient with respect to the rotated rows, rotated
 *                 by -t, is the gradient with respect to the rows (hstu_attn_bwd's dq and dk).
 *   q_out, k_out  device bf16 [rows, H, d], rows q_out_ld / k_out_ld apart.  Each may be its own
 *                 input (in place, same stride); otherwise no output may overlap another tensor.
 * Errors: HSTU_ERR_INVALID_ARGUMENT (NULL pointers, sizes, sections, overlap), HSTU_ERR_UNSUPPORTED
 * (d, pairs, strides or alignment), HSTU_ERR_CUDA.
 */
hstu_status_t hstu_rotary(const void* q, int64_t q_ld, const void* k, int64_t k_ld,
                          const hstu_rotation_t* rotation, int32_t inverse,
                          int32_t H, int32_t d, int32_t rows,
                          void* q_out, int64_t q_out_ld, void* k_out, int64_t k_out_ld, void* stream);

/*
 * hstu_paged_append — writes every user's new K and V rows to their places in the cache.
 *   q, k, v       device bf16 [total_new, H, d], rows *_ld elements apart.  q may be NULL.
 *   rotation      NULL: K is copied as it is, and q must be NULL.  Otherwise K and q are rotated.
 *   cache         see above; the pages that receive rows must belong to one user only, and stand once
 *                 in its table.  No other row of the cache is touched.  K and V may interleave, but no
 *                 element may be of both, nor of two rows, heads or pages of one (INVALID_ARGUMENT):
 *                 of the strides, each is at least the extent of what the smaller ones reach.
 *   q_offsets     device int32 [B+1], q_offsets[0] = 0, non-decreasing, q_offsets[B] = total_new.
 *   kv_len        device int32 [B], kv_len[b] >= n_b: lengths after the call.
 *   q_out         device bf16 [total_new, H, d], the rotated q (may be q itself); NULL with q.
 * Errors on the host as for hstu_rotary (also: a token tensor that overlaps the cache).  On the device,
 * HSTU_ERR_BAD_OFFSETS is reported for inconsistent offsets or lengths (the user's rows are skipped)
 * and for a table entry outside the pool (the rows of that page are not written).
 */
hstu_status_t hstu_paged_append(const void* q, int64_t q_ld, const void* k, int64_t k_ld,
                                const void* v, int64_t v_ld,
                                const hstu_rotation_t* rotation, const hstu_paged_cache_t* cache,
                                const int32_t* q_offsets, const int32_t* kv_len,
                                int32_t B, int32_t H, int32_t d, int32_t total_new,
                                void* q_out, int64_t q_out_ld, void* stream);

/*
 * hstu_paged_attn_fwd — hstu_attn_fwd_cached over the paged cache: each user's new rows attend to its
 * kv_len[b] cached rows, which include the new ones (hstu_paged_append has written them).
 *
 *     out[i,h,:] = (1/N) * sum_{j in A(i)} silu(alpha * <q[i,h,:], k[j,h,:]>) * v[j,h,:]
 *
 * with A(i) as in hstu_attn.h: the last num_targets[b] of the new rows are candidates, which see the
 * history and themselves; the others are history and see what precedes them and themselves.  A row
 * always sees itself, so no row is empty.
 *   q             device bf16 [total_new, H, d], rows q_ld elements apart; d in {32, 64, 128}.
 *   cache         see above; read only.
 *   q_offsets, kv_len   as in hstu_paged_append.
 *   num_targets   device int32 [B], 0 <= T_b <= n_b; NULL means none.
 *   max_new, max_kv     upper bounds on every n_b and kv_len[b] (they choose the kernel and its launch
 *                 shape; a user beyond them is reported as HSTU_ERR_BAD_OFFSETS and skipped).
 *   alpha, N      as in hstu_attn_fwd.
 *   out           device bf16 [total_new, H, d], rows out_ld apart; may overlap neither q nor the cache.
 * A call that needs a workspace takes it from the library's pool, as in hstu_attn.h (captured into a graph,
 * the graph owns it): 48 bytes for each head and 128 rows (and each head and user), and where few items may
 * be cut, 512 * d bytes for each piece they may be cut into, at most 4 for each SM (38 MB at d = 128).  With up
 * to 16 rows a user: none, or 256 * d bytes for each SM.
 * K, V and q must be finite in the rows that a user owns: a tile's masked pairs get the weight zero, but
 * zero times an infinite V of the same user is not zero.  Nothing else in the cache needs to be:
 * rows behind a user's last one may hold anything.
 * Errors on the host as in hstu_paged_append.  On the device, HSTU_ERR_BAD_OFFSETS for inconsistent
 * offsets or lengths (the user's rows of out are not written) and for a table entry outside the pool
 * (its rows count as zeros).
 */
hstu_status_t hstu_paged_attn_fwd(const void* q, int64_t q_ld, const hstu_paged_cache_t* cache,
                                  const int32_t* q_offsets, const int32_t* kv_len,
                                  const int32_t* num_targets, int32_t B, int32_t H, int32_t d,
                                  int32_t total_new, int32_t max_new, int32_t max_kv,
                                  float alpha, float N, void* out, int64_t out_ld, void* stream);

/*
 * hstu_paged_selfcheck_fwd_timeout — hstu_attn_selfcheck_fwd_timeout for the paged kernel: the work of
 * hstu_paged_attn_fwd on the kernel for many rows, with every pipeline wait limited to limit_ns
 * nanoseconds (1 .. 1e9).  A wait that runs out is reported as HSTU_ERR_TIMEOUT, the kernel drains what
 * it started and returns, and the context stays usable; `out` is left partly written.
 */
hstu_status_t hstu_paged_selfcheck_fwd_timeout(const void* q, int64_t q_ld, const hstu_paged_cache_t* cache,
                                               const int32_t* q_offsets, const int32_t* kv_len,
                                               const int32_t* num_targets, int32_t B, int32_t H, int32_t d,
                                               int32_t total_new, int32_t max_new, int32_t max_kv,
                                               float alpha, float N, void* out, int64_t out_ld,
                                               uint64_t limit_ns, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* HSTU_PAGED_H_ */
