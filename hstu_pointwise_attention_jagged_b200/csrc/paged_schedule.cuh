// paged_schedule.cuh — work plan of the many-row paged attention (the paged form of hstu_fwd_kernel).
//
// The unit of work is a piece: some consecutive key tiles of one item (user, head, 128 query rows), taken
// from a queue by the CTAs.  With many items every piece is a whole item, in waves of users whose
// K and V fit a quarter of L2, by non-increasing cost within a wave (schedule.cuh).  With few items for the
// CTAs, whole items can leave SMs idle: 192 items of 26 tiles on 148 SMs take the time of 52 tiles, where
// 34 would do.  So the plan may cut items into pieces of at most q tiles, choosing q by the
// estimate rounds * (q + overhead).  The pieces of a cut item leave fp32 partial outputs, and the last one to
// finish adds them up in order (hstu_fwd_sm100.cuh, epilogue).  Pieces of one key range of one user and head
// are neighbours in the queue: CTAs that work side by side read the same K and V.
#pragma once

#include <climits>
#include <cstdint>

#include "paged_cache.cuh"
#include "schedule.cuh"

namespace hstu {

constexpr int kMaxCutRounds = 4;  // cut items make at most this many pieces for each CTA
constexpr int kMaxCuts = 16;      // pieces of the longest item
constexpr int kMinPieceTiles = 2;
constexpr int kPieceOverhead = 3; // tiles: filling the pipeline, writing and adding the partial

struct PagedSchedArgs {
  PagedView cache;
  const int32_t* q_offsets;
  const int32_t* kv_len;
  const int32_t* num_targets;
  int32_t B, H, total_new, max_new, max_kv, nbins, nwaves, wave_rows, num_ctas, max_items, max_cut;  // max_items: H * (total_new / 128 + B)
  PagedPlan plan;
  unsigned* err;
};

// One CTA of kSchedThreads threads.
__global__ void __launch_bounds__(kSchedThreads) paged_schedule_kernel(const PagedSchedArgs a) {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  __shared__ int hist[kMaxCostBins];
  __shared__ long long scan_scratch[2][32];
  __shared__ long long carry_blocks, carry_rows;
  __shared__ int first_bad;  // first user whose offsets decrease
  __shared__ int longest, pieces_of[kMaxCuts + 1];
  __shared__ PagedUser s_user[kCachedUsers];
  __shared__ int s_start[kCachedUsers + 1], s_wave[kCachedUsers], s_cost[kCachedUsers];
  const bool cached = a.B <= kCachedUsers;
  const int tid = threadIdx.x;
  if (tid == 0) {
    carry_blocks = 0;
    carry_rows = 0;
    longest = 0;
    first_bad = INT_MAX;
  }
  if (tid <= kMaxCuts) pieces_of[tid] = 0;
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
      if (a.q_offsets[b + 1] < u.q0) atomicMin(&first_bad, b);
    }
    __syncthreads();
    if (b < a.B) {
      // Behind decreasing offsets users may overlap, and their blocks be more than the plan has room for.
      if (!u.ok || b >= first_bad) u.n = u.L = 0;
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
        s_cost[b] = 0;
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
  const int items = nblocks * a.H;  // at most a.max_items
  // Block g: its user, index within the user and tiles.
  auto block_of = [&](int g, int& b, int& blk) {
    b = owner_of(cached ? s_start : a.plan.block_start, a.B, g);
    blk = g - (cached ? s_start[b] : a.plan.block_start[b]);
    const PagedUser u = cached ? s_user[b]
                               : paged_user(a.cache, a.q_offsets, a.kv_len, a.num_targets, b, a.total_new, a.max_new,
                                            a.max_kv);
    const int rows = u.n - blk * kItemRows;
    return item_cost(u.L - u.n + blk * kItemRows, rows < kItemRows ? rows : kItemRows, u.L - u.T);
  };

  // Cuts that can be tried: c pieces of every item may not be more than there is room for.
  const int most = items > 0 ? min(kMaxCuts, a.max_cut / items) : 1;
  if (cached && most > 1) {
    // Most tiles of an item, for each user (s_cost) and in all.
    for (int g = tid; g < nblocks; g += kSchedThreads) {
      int b, blk;
      const int cost = block_of(g, b, blk);
      atomicMax(&s_cost[b], cost);
      atomicMax(&longest, cost);
    }
    __syncthreads();
    // Pieces when the longest item is cut in c.
    const int top = longest;
    if (tid < a.B && s_cost[tid] > 0) {
      const int rows = (s_start[tid + 1] - s_start[tid]) * a.H;
      for (int c = 1; c <= most; ++c) atomicAdd(&pieces_of[c], rows * cdiv(s_cost[tid], cdiv(top, c)));
    }
    __syncthreads();
    // The best c by estimated time, ties to the smaller: lane c - 1 of each warp rates c.
    int best = (tid & 31) + 1, time = INT_MAX;
    if (best <= most && best <= top && pieces_of[best] <= a.max_cut) {
      const int q = cdiv(top, best);
      if (best == 1 || q >= kMinPieceTiles)
        time = cdiv(pieces_of[best], a.num_ctas) * (q + (best > 1 ? kPieceOverhead : 0));
    }
    for (int o = 16; o > 0; o >>= 1) {
      const int t2 = __shfl_xor_sync(0xffffffffu, time, o), b2 = __shfl_xor_sync(0xffffffffu, best, o);
      if (t2 < time || (t2 == time && b2 < best)) {
        time = t2;
        best = b2;
      }
    }
    if (best > 1) {
      // Queue places: user, head, part, block.  Every item of a user is cut alike; the places of parts
      // that a short item does not have stay empty.
      const int q = cdiv(top, best);
      long long mine = 0, tot;
      if (tid < a.B) mine = (long long)(s_start[tid + 1] - s_start[tid]) * a.H * cdiv(s_cost[tid], q);
      const int first = (int)(block_inclusive_scan(mine, scan_scratch[0], &tot) - mine);
      if (tid < a.B) hist[tid] = first;
      __syncthreads();
      for (int x = tid; x < nblocks * a.H; x += kSchedThreads) {
        PagedPiece p;
        p.h = x / nblocks;
        const int cost = block_of(x - p.h * nblocks, p.b, p.block);
        const int parts = cdiv(s_cost[p.b], q);
        p.pitch = s_start[p.b + 1] - s_start[p.b];
        p.parts = min(parts, cost);
        const int at = hist[p.b] + p.h * parts * p.pitch + p.block;
        for (p.part = 0; p.part < parts; ++p.part) {
          p.tile0 = p.part < p.parts ? cost * p.part / p.parts : 0;
          p.tiles = p.part < p.parts ? cost * (p.part + 1) / p.parts - p.tile0 : 0;
          a.plan.pieces[at + p.part * p.pitch] = p;
        }
        for (int k = 0; k < 4; ++k) a.plan.done[at * 4 + k] = 0;
      }
      if (tid == 0) {
        a.plan.header[0] = 0;
        a.plan.header[1] = (int)tot;
        a.plan.header[2] = 0;
        a.plan.header[3] = best;
      }
      return;
    }
  }

  // Whole items, as schedule_kernel: a counting sort of the blocks by (wave, non-increasing cost).
  const long long waves = (carry_rows + a.wave_rows - 1) / a.wave_rows;  // that the batch reaches
  const int nkeys = a.nbins * (int)(cached && waves < a.nwaves ? (waves > 0 ? waves : 1) : a.nwaves);
  for (int i = tid; i < nkeys; i += kSchedThreads) hist[i] = 0;
  __syncthreads();
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
    p.tile0 = 0;
    p.tiles = cost;
    p.parts = 1;
    p.part = p.pitch = 0;
    const int pos = atomicAdd(&hist[key_of(p.b, cost)], a.H);
    for (p.h = 0; p.h < a.H; ++p.h)
      if (pos + p.h < items) a.plan.pieces[pos + p.h] = p;
  }
  if (tid == 0) {
    a.plan.header[0] = 0;
    a.plan.header[1] = items;
    a.plan.header[2] = 0;
    a.plan.header[3] = 1;
  }
}

}  // namespace hstu
