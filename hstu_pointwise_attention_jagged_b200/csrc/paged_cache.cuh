// paged_cache.cuh — device view of the paged K/V cache (hstu_paged_cache_t), the checks of one user's
// lengths that every kernel on it makes, and the work plan of the many-row attention.
#pragma once

#include <cstdint>
#include <cuda_bf16.h>

namespace hstu {

struct PagedView {
  __nv_bfloat16* k;
  __nv_bfloat16* v;
  int64_t page_stride, row_stride, head_stride;  // elements
  int32_t num_pages, page_shift;                 // page_size = 1 << page_shift
  const int32_t* table;
  int32_t table_width;
  int64_t table_ld;
};

// New rows [q0, q0 + n) of the packed tensors, L rows in the cache with them, T candidates at the end.
struct PagedUser {
  int32_t q0, n, L, T;
  bool ok;
};

// Reads and checks user b.  `ok` false: nothing of the user may be read or written.  kv_len is not
// bounded by max_kv when max_kv < 0.
__device__ __forceinline__ PagedUser paged_user(const PagedView& c, const int32_t* q_offsets, const int32_t* kv_len,
                                                const int32_t* num_targets, int b, int total_new, int max_new,
                                                int max_kv) {
  PagedUser u;
  u.q0 = q_offsets[b];
  const int o1 = q_offsets[b + 1];
  u.L = kv_len[b];
  u.T = num_targets ? num_targets[b] : 0;
  u.ok = u.q0 >= 0 && o1 >= u.q0 && o1 <= total_new;
  u.n = u.ok ? o1 - u.q0 : 0;
  // Pages are looked up only for users with new rows.
  u.ok = u.ok && u.L >= u.n && u.T >= 0 && u.T <= u.n && u.n <= max_new && (max_kv < 0 || u.L <= max_kv) &&
         (u.n == 0 || ((static_cast<int64_t>(u.L) + (1 << c.page_shift) - 1) >> c.page_shift) <= c.table_width);
  return u;
}

// A piece of work of the many-row attention: key tiles [tile0, tile0 + tiles) of an item's (user b, head h,
// `nrows` query rows from row q_row0 of q, at positions pos0 on of a user with L rows, U of them
// history).  tiles = 0: nothing to do.
struct PagedPiece {
  int32_t b, h, q_row0, pos0;
  int32_t nrows, L, U, tile0;
  int32_t tiles, parts, part, pitch;  // parts: pieces of the item (1: whole); part: which one this is;
                                      // pitch: queue places between the item's pieces
};
static_assert(sizeof(PagedPiece) == 48, "three 16-byte loads");

struct PagedPlan {
  int32_t* header;       // [4] {pieces taken beyond the CTAs' first ones, pieces, whole items before the cut, 0}
  int32_t* block_start;  // [B+1] first block of each user
  int32_t* done;         // [4 * max_cut] finished pieces of a cut item, for each quarter of its rows
  PagedPiece* pieces;    // [max_pieces] the queue
};

// The paged form of the forward kernel's parameters.
struct PagedFwd {
  PagedView cache;
  PagedPlan plan;
  float4* partials;  // [place among the cut pieces][D / 4][128 rows]: their fp32 sums
};

}  // namespace hstu
