// paged_schedule.cuh — work plan of the many-row paged attention (the paged form of hstu_fwd_kernel).
//
// The unit of work is a piece: some consecutive key tiles of one item (user, head, 128 query rows).
// Two forms, chosen on the device from the number of items:
//   queue    many items for the CTAs: every piece is a whole item, taken from a queue in waves of users
//            whose K and V fit a quarter of L2, by non-increasing cost within a wave (schedule.cuh).
//   ranges   few items: the tiles of all items, in item order, are dealt out in equal runs, one for each CTA,
//            and an item that a boundary falls into is cut there.  Whole items would leave SMs
//            idle: 192 items of 26 tiles on 148 SMs take 52 tiles' time, the runs take 34.  The
//            pieces of a cut item leave fp32 partial outputs, and the last one to finish adds them
//            up in piece order (hstu_fwd_sm100.cuh, epilogue).
#pragma once

#include <climits>
#include <cstdint>

#include "paged_cache.cuh"
#include "schedule.cuh"

namespace hstu {

constexpr int kRangeItemsPerCta = 8;    // fewer items than this for each CTA: ranges
constexpr int kMaxRangeItems = 2048;    // ... if the items fit the tables below
constexpr int kMinRangeTiles = 4;       // a run is at least this long (the sums of a shorter one cost more than it does)

struct PagedSchedArgs {
  PagedView cache;
  const int32_t* q_offsets;
  const int32_t* kv_len;
  const int32_t* num_targets;
  int32_t B, H, total_new, max_new, max_kv, nbins, nwaves, wave_rows, num_ctas, max_pieces;
  PagedPlan plan;
  unsigned* err;
};

// First tile of range r when `tiles` tiles are dealt out in `ranges` runs; ranges <= tiles, so none is empty.
__device__ __forceinline__ int range_begin(int tiles, int ranges, int r) {
  return (int)((int64_t)tiles * r / ranges);
}
// Range that tile x falls into.
__device__ __forceinline__ int range_of(int tiles, int ranges, int x) {
  int r = (int)((int64_t)x * ranges / tiles);
  while (r + 1 < ranges && range_begin(tiles, ranges, r + 1) <= x) ++r;
  while (r > 0 && range_begin(tiles, ranges, r) > x) --r;
  return r;
}

// One CTA of kSchedThreads threads.
__global__ void __launch_bounds__(kSchedThreads) paged_schedule_kernel(const PagedSchedArgs a) {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  __shared__ int hist[kMaxCostBins];
  __shared__ int cum[kMaxRangeItems];
  __shared__ long long scan_scratch[2][32];
  __shared__ long long carry_blocks, carry_rows;
  __shared__ int slots;
  __shared__ PagedUser s_user[kCachedUsers];
  __shared__ int s_start[kCachedUsers + 1], s_wave[kCachedUsers];
  const bool cached = a.B <= kCachedUsers;
  const int tid = threadIdx.x;
  if (tid == 0) {
    carry_blocks = 0;
    carry_rows = 0;
    slots = 0;
  }
  for (int i = tid; i < kMaxCostBins; i += kSchedThreads) hist[i] = 0;
  __syncthreads();

  // Pass 1: check every user; prefix sums of 128-row blocks and of cached rows.
  for (int base = 0; base < a.B; base += kSchedThreads) {
    const int b = base + tid;
    long long blocks = 0, rows = 0;
    PagedUser u;
    if (b < a.B) {
      u = paged_user(a.cache, a.q_offsets, a.kv_len, a.num_targets, b, a.total_new, a.max_new, a.max_kv);
      bool bad = !u.ok;
      if (b == 0) bad |= u.q0 != 0;
      if (b == a.B - 1) bad |= a.q_offsets[a.B] != a.total_new;
      if (bad) atomicOr(a.err, kErrBadOffsets);
      if (!u.ok) u.n = u.L = 0;
      blocks = cdiv(u.n, kItemRows);
      rows = u.n > 0 ? u.L : 0;
    }
    long long incl_b = blocks, incl_r = rows, tot_b, tot_r;
    block_inclusive_scan2(incl_b, incl_r, scan_scratch, tot_b, tot_r);
    if (b < a.B) {
      const int start = (int)(carry_blocks + incl_b - blocks);
      const long long wave = (carry_rows + incl_r - rows) / a.wave_rows;
      a.plan.block_start[b] = start;
      if (cached) {
        s_user[b] = u;
        s_start[b] = start;
        s_wave[b] = (int)(wave < a.nwaves ? wave : a.nwaves - 1);
      }
    }
    __syncthreads();
    if (tid == 0) {
      carry_blocks += tot_b;
      carry_rows += tot_r;
    }
    __syncthreads();
  }
  const int nblocks = (int)carry_blocks;
  if (tid == 0) {
    a.plan.block_start[a.B] = nblocks;
    if (cached) s_start[a.B] = nblocks;
  }
  __syncthreads();
  // Block g: its user, index within the user and tiles.  Overlapping (inconsistent) offsets can make
  // the users' blocks more than the plan has room for; the surplus is dropped, and was reported.
  const int64_t items64 = (int64_t)nblocks * a.H;
  const int items = (int)(items64 < a.max_pieces - a.num_ctas ? items64 : a.max_pieces - a.num_ctas);
  auto block_of = [&](int g, int& b, int& blk) {
    b = owner_of(cached ? s_start : a.plan.block_start, a.B, g);
    blk = g - (cached ? s_start[b] : a.plan.block_start[b]);
    const PagedUser u = cached ? s_user[b]
                               : paged_user(a.cache, a.q_offsets, a.kv_len, a.num_targets, b, a.total_new, a.max_new,
                                            a.max_kv);
    const int rows = u.n - blk * kItemRows;
    return item_cost(u.L - u.n + blk * kItemRows, rows < kItemRows ? rows : kItemRows, u.L - u.T);
  };

  if (items < kRangeItemsPerCta * a.num_ctas && items <= kMaxRangeItems &&
      (int64_t)items * (a.max_kv / kTileRows + 2) < INT_MAX) {
    // ------------------------------------------------------------------ ranges
    // Items in the order (user, head, block): neighbours read the same K and V.
    auto item_of = [&](int i, int& b, int& blk, int& h) {
      // The user's first item is H times its first block; within it heads, then blocks.
      b = owner_of(cached ? s_start : a.plan.block_start, a.B, i / a.H);
      const int s0 = cached ? s_start[b] : a.plan.block_start[b], s1 = cached ? s_start[b + 1] : a.plan.block_start[b + 1];
      const int in = i - s0 * a.H;
      h = in / (s1 - s0);
      blk = in - h * (s1 - s0);
      int b2, blk2;
      return block_of(s0 + blk, b2, blk2);
    };
    int total = 0;
    for (int base = 0; base < items; base += kSchedThreads) {
      int b, blk, h;
      long long cost = base + tid < items ? item_of(base + tid, b, blk, h) : 0, tot;
      const long long incl = block_inclusive_scan(cost, scan_scratch[0], &tot);
      if (base + tid < items) cum[base + tid] = total + (int)incl;
      total += (int)tot;
    }
    __syncthreads();
    const int most = total / kMinRangeTiles;
    const int ranges = most < 1 ? 1 : (most < a.num_ctas ? most : a.num_ctas);
    int pieces = 0;
    for (int base = 0; base < items; base += kSchedThreads) {
      const int i = base + tid;
      int c0 = 0, c1 = 0, r0 = 0, parts = 0;
      if (i < items) {
        c0 = i > 0 ? cum[i - 1] : 0;
        c1 = cum[i];
        r0 = range_of(total, ranges, c0);
        parts = range_of(total, ranges, c1 - 1) - r0 + 1;
      }
      long long tot;
      const int first = pieces + (int)block_inclusive_scan(parts, scan_scratch[0], &tot) - parts;
      pieces += (int)tot;
      if (i < items) {
        PagedPiece p;
        item_of(i, p.b, p.block, p.h);
        p.parts = parts;
        p.slot = parts > 1 ? atomicAdd(&slots, parts) : 0;  // any order: a slot only names a place
        for (int k = 0; k < parts; ++k) {
          const int lo = max(c0, range_begin(total, ranges, r0 + k));
          const int hi = r0 + k + 1 < ranges ? min(c1, range_begin(total, ranges, r0 + k + 1)) : c1;
          p.tile0 = lo - c0;
          p.tiles = hi - lo;
          p.part = k;
          a.plan.pieces[first + k] = p;
          if (lo == range_begin(total, ranges, r0 + k)) a.plan.starts[r0 + k] = first + k;
        }
        if (parts > 1)
          for (int q = 0; q < 4; ++q) a.plan.done[p.slot * 4 + q] = 0;
      }
    }
    __syncthreads();
    if (tid == 0) {
      a.plan.starts[ranges] = pieces;
      a.plan.header[0] = 0;
      a.plan.header[1] = pieces;
      a.plan.header[2] = 0;
      a.plan.header[3] = items > 0 ? ranges : 0;
      a.plan.header[4] = slots;
    }
    return;
  }

  // -------------------------------------------------------------------- queue
  // As schedule_kernel: a counting sort of the blocks by (wave, non-increasing cost).
  const int nkeys = a.nbins * a.nwaves;
  auto key_of = [&](int b, int cost) {
    int wave = 0;
    if (cached) wave = s_wave[b];
    else wave = (int)((int64_t)b * a.nwaves / a.B);  // large batches: by the user's index
    return wave * a.nbins + (a.nbins - 1 - (cost < a.nbins ? cost : a.nbins - 1));
  };
  for (int g = tid; g < nblocks; g += kSchedThreads) {
    int b, blk;
    const int cost = block_of(g, b, blk);
    atomicAdd(&hist[key_of(b, cost)], a.H);
  }
  __syncthreads();
  const int per = cdiv(nkeys, kSchedThreads);
  long long part = 0;
  for (int k = 0; k < per; ++k)
    if (tid * per + k < nkeys) part += hist[tid * per + k];
  __syncthreads();
  long long tot;
  long long run = block_inclusive_scan(part, scan_scratch[0], &tot) - part;
  for (int k = 0; k < per; ++k) {
    const int key = tid * per + k;
    if (key < nkeys) {
      const int n = hist[key];
      hist[key] = (int)run;
      run += n;
    }
  }
  __syncthreads();
  for (int g = tid; g < nblocks; g += kSchedThreads) {
    PagedPiece p;
    const int cost = block_of(g, p.b, p.block);
    p.parts = 1;
    p.tile0 = 0;
    p.tiles = cost;
    p.slot = p.part = 0;
    const int pos = atomicAdd(&hist[key_of(p.b, cost)], a.H);
    for (p.h = 0; p.h < a.H; ++p.h)
      if (pos + p.h < items) a.plan.pieces[pos + p.h] = p;
  }
  if (tid == 0) {
    a.plan.header[0] = 0;
    a.plan.header[1] = items;
    a.plan.header[2] = 0;
    a.plan.header[3] = 0;
    a.plan.header[4] = 0;
  }
}

}  // namespace hstu
