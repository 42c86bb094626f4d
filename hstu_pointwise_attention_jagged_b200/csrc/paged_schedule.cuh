// paged_schedule.cuh — work plan of the many-row paged attention (the paged form of hstu_fwd_kernel).
//
// The unit of work is a piece: some consecutive key tiles of one item (user, head, 128 query rows), taken
// from a queue by the CTAs.  With many items every piece is a whole item, in waves of users whose
// K and V fit a quarter of L2, by non-increasing cost within a wave (schedule.cuh).  With few items for the
// CTAs, whole items can leave SMs idle: 192 items of 26 tiles on 148 SMs take the time of 52 tiles, where
// 34 would do.  So the plan may cut the items of the first users into pieces of at most q tiles and put them behind
// the others' whole items, where they fill the last round; it chooses both numbers by an estimate of the
// time.  The pieces of a cut item leave fp32 partial outputs, and the last one to finish adds them up in order
// (hstu_fwd_sm100.cuh, epilogue).  Pieces of one key range of one user and head are neighbours in the queue:
// CTAs that work side by side read the same K and V.  (us, H = 4, d = 128: 16 users x 300 rows of 3300, whole items
// 60.9, all items in halves 59.2, 4 users' in thirds 54.8; 5 x 1000 of 5000, whole 74.3, all in thirds 70.1, one
// user's in quarters 65.2; 20 ragged users of up to 300 rows over 1500, all in pieces 30.6, some 24.3.)
//
// The plan is one CTA's work between two kernels, so what it costs is latency, much of it fetching
// instructions that run once: loops are not unrolled, the block scan is one function, 64-bit divisions are
// avoided, and each block's cost is computed once and kept on chip.
#pragma once

#include <climits>
#include <cstdint>

#include "paged_cache.cuh"
#include "schedule.cuh"

namespace hstu {

constexpr int kMaxCutRounds = 4;  // cut items make at most this many pieces for each CTA
constexpr int kMaxRounds = 4;     // batches of more whole items for each CTA are not cut
constexpr int kMaxCuts = 16;      // pieces of the longest item
constexpr int kMinPieceTiles = 2;
// Fitted to measured times, in tiles (1.2 us at d = 128): what a whole item and a piece take beyond their own, and
// what the last addition takes for each part of an item.  A cut has to promise kCutGain of the time.  The same
// figures serve d = 64 and 32, where a tile takes some 0.85 us and a partial is smaller; one of the shapes compared
// lost by it (6 ragged users, 8 heads, d = 64: 43.2 -> 45.1 us against cutting all items or none).
constexpr float kItemOverhead = 1.0f, kPieceOverhead = 2.0f, kPartAdd = 1.2f, kCutGain = 0.08f;
constexpr int kCachedBlocks = 2048;  // batches up to this many 128-row blocks keep their costs in shared memory

struct PagedSchedArgs {
  PagedView cache;
  const int32_t* q_offsets;
  const int32_t* kv_len;
  const int32_t* num_targets;
  int32_t B, H, total_new, max_new, max_kv, wave_rows, num_ctas, max_cut;
  PagedPlan plan;
  unsigned* err;
};

// Inclusive prefix sum over the CTA of one value a thread (or two, in the halves of 64 bits); *total gets
// the sum.  scratch: kSchedWarps values.
template <typename T>
static __device__ __noinline__ T paged_scan(T v, T* scratch, T* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const T n = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += n;
  }
  if (lane == 31) scratch[warp] = v;
  __syncthreads();
  T sum = 0;
#pragma unroll
  for (int w = 0; w < kSchedWarps; ++w) {
    if (w < warp) v += scratch[w];
    sum += scratch[w];
  }
  *total = sum;
  __syncthreads();
  return v;
}

// Block g of a user: its rows and tiles.
__device__ __forceinline__ int block_rows(const PagedUser& u, int blk) { return min(u.n - blk * kItemRows, kItemRows); }
__device__ __forceinline__ int block_cost(const PagedUser& u, int blk) {
  return item_cost(u.L - u.n + blk * kItemRows, block_rows(u, blk), u.L - u.T);
}

// One CTA of kSchedThreads threads.
__global__ void __launch_bounds__(kSchedThreads) paged_schedule_kernel(const PagedSchedArgs a) {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  __shared__ __align__(16) int hist[kMaxCostBins];
  __shared__ unsigned long long scratch2[kSchedWarps];
  __shared__ int scratch[kSchedWarps];
  __shared__ int first_bad;  // first user whose offsets decrease
  __shared__ int longest, all_tiles;
  __shared__ int2 s_choice[kSchedWarps];
  __shared__ PagedUser s_user[kCachedUsers];
  __shared__ int s_start[kCachedUsers + 1], s_tiles[kCachedUsers], s_cost[kCachedUsers];
  __shared__ unsigned s_block[kCachedBlocks];  // user | cost << 8
  static_assert(kCachedUsers <= 256, "a user in 8 bits");
  const int tid = threadIdx.x;
  if (tid == 0) {
    longest = all_tiles = 0;
    first_bad = INT_MAX;
  }
  for (int i = tid; i < kMaxCostBins / 4; i += kSchedThreads) reinterpret_cast<int4*>(hist)[i] = make_int4(0, 0, 0, 0);
  const bool few_users = a.B <= kCachedUsers;
  auto user = [&](int b) {
    return paged_user(a.cache, a.q_offsets, a.kv_len, a.num_targets, b, a.total_new, a.max_new, a.max_kv);
  };
  asm volatile("griddepcontrol.wait;" ::: "memory");
  __syncthreads();

  // Pass 1: check every user; prefix sums of 128-row blocks (low half) and, for the waves, of key tiles.
  unsigned long long carry = 0;
#pragma unroll 1
  for (int base = 0; base < a.B; base += kSchedThreads) {
    const int b = base + tid;
    unsigned long long mine = 0;
    PagedUser u;
    if (b < a.B) {
      u = user(b);
      const int next = a.q_offsets[b + 1];
      if (!u.ok || (b == 0 && u.q0 != 0) || (b == a.B - 1 && next != a.total_new)) atomicOr(a.err, kErrBadOffsets);
      if (next < u.q0) atomicMin(&first_bad, b);
    }
    __syncthreads();
    if (b < a.B) {
      // Behind decreasing offsets users may overlap, and their blocks be more than the plan has room for.
      if (!u.ok || b >= first_bad) u.n = u.L = 0;
      const int tiles = u.n > 0 ? min(u.L / kTileRows, 1 << 22) : 0;  // the sum of kCachedUsers fits 31 bits
      mine = (unsigned)cdiv(u.n, kItemRows) | (unsigned long long)tiles << 32;
    }
    unsigned long long all;
    const unsigned long long upto = carry + paged_scan(mine, scratch2, &all) - mine;
    carry += all;
    if (b < a.B) {
      const int start = (int)(unsigned)upto;
      a.plan.block_start[b] = start;
      if (few_users) {
        s_user[b] = u;
        s_start[b] = start;
        s_tiles[b] = (int)(upto >> 32);
        s_cost[b] = 0;
      }
    }
  }
  const int nblocks = (int)(unsigned)carry;  // times H: at most the plan's room, H * (total_new / 128 + B)
  if (tid == 0) {
    a.plan.block_start[a.B] = nblocks;
    if (few_users) s_start[a.B] = nblocks;
  }
  __syncthreads();

  // Pass 2: every block's tiles.
  const bool cached = few_users && nblocks <= kCachedBlocks;
  auto start_of = [&](int b) { return few_users ? s_start[b] : a.plan.block_start[b]; };
  auto owner = [&](int g) { return few_users ? owner_of(s_start, a.B, g) : owner_of(a.plan.block_start, a.B, g); };
  auto known = [&](int b) { return few_users ? s_user[b] : user(b); };
  int most_tiles = 0, sum_tiles = 0;
#pragma unroll 1
  for (int g = tid; g < nblocks; g += kSchedThreads) {
    const int b = owner(g), cost = block_cost(known(b), g - start_of(b));
    most_tiles = max(most_tiles, cost);
    sum_tiles += min(cost, 1 << 19);  // only an estimate; kCachedBlocks of them fit
    if (cached) {
      s_block[g] = (unsigned)b | (unsigned)cost << 8;
      atomicMax(&s_cost[b], cost);
    }
  }
  most_tiles = __reduce_max_sync(0xffffffffu, most_tiles);
  sum_tiles = __reduce_add_sync(0xffffffffu, sum_tiles);
  if ((tid & 31) == 0) {
    atomicMax(&longest, most_tiles);
    atomicAdd(&all_tiles, sum_tiles);
  }
  __syncthreads();
  const int top = longest;
  auto block_of = [&](int g, int& b, int& blk, int& cost) {
    if (cached) {
      b = (int)(s_block[g] & 255u);
      cost = (int)(s_block[g] >> 8);
    } else {
      b = owner(g);
      cost = -1;
    }
    blk = g - start_of(b);
    if (cost < 0) cost = block_cost(known(b), blk);
  };
  auto piece_of = [&](int b, int blk, int cost) {
    const PagedUser u = known(b);
    PagedPiece p;
    p.b = b;
    p.q_row0 = u.q0 + blk * kItemRows;
    p.pos0 = u.L - u.n + blk * kItemRows;
    p.nrows = block_rows(u, blk);
    p.L = u.L;
    p.U = u.L - u.T;
    p.tile0 = 0;
    p.tiles = cost;
    p.parts = 1;
    p.part = p.pitch = 0;
    return p;
  };
  auto put = [&](int at, const PagedPiece& p) {
    int4* to = reinterpret_cast<int4*>(a.plan.pieces + at);
    to[0] = make_int4(p.b, p.h, p.q_row0, p.pos0);
    to[1] = make_int4(p.nrows, p.L, p.U, p.tile0);
    to[2] = make_int4(p.tiles, p.parts, p.part, p.pitch);
  };

  // The cut: the items of the first `cut_users` users in pieces of at most q tiles, behind the whole items of
  // the others in the queue, or none.
  const int items = nblocks * a.H;
  int cut_users = 0, q = 1, cut_places = 0;
  const int most = items > 0 ? min(kMaxCuts, top / kMinPieceTiles) : 1;
  if (cached && most > 1 && nblocks <= kMaxRounds * a.num_ctas / a.H) {
    // Estimated time: rounds of whole items at their mean cost, then rounds of pieces, some of which the CTAs
    // without an item in the last whole round have taken; no less than the longest item, nor than all of
    // the work spread evenly.
    const float mean = (float)all_tiles / nblocks + kItemOverhead, even = mean * items, each = 1.0f / a.num_ctas;
    auto rounds_of = [&](float n) { return ceilf(n * each - 1e-3f); };
    auto estimate = [&](int whole, int pieces, float size) {  // size: with the overhead
      const float rounds = rounds_of((float)whole), idle = rounds * a.num_ctas - whole;
      const float left = fmaxf((float)pieces - idle * floorf(__fdividef(mean, size)), 0.0f);
      const float time = rounds * mean + rounds_of(left) * size;
      return fmaxf(fmaxf(time, whole > 0 ? (float)top : 0.0f), (even + pieces * kPieceOverhead) * each);
    };
    float least = estimate(items, 0, 1.0f) * (1.0f - kCutGain);
    int choice = 0;  // users | c << 16
    if (even * each + 2.0f * kPartAdd < least) {  // else nothing can reach it
      // A half warp tries the numbers of users for each q, top / 1 to top / kMaxCuts, in sixteen steps.
      constexpr int kEach = kSchedThreads / kMaxCuts;
      static_assert(kEach == 16, "a half warp each");
      const int c = tid / kEach + 1, lane = tid % kEach, size = cdiv(top, c), step = cdiv(a.B, kEach);
      const int users = min((lane + 1) * step, a.B);
      int n = 0;
#pragma unroll 1
      for (int b = lane * step; b < users; ++b) n += (s_start[b + 1] - s_start[b]) * a.H * cdiv(s_cost[b], size);
#pragma unroll
      for (int o = 1; o < kEach; o <<= 1) {
        const int up = __shfl_up_sync(0xffffffffu, n, o, kEach);
        if (lane >= o) n += up;
      }
      if (c > 1 && c <= most && n <= a.max_cut) {
        const float time = estimate((nblocks - s_start[users]) * a.H, n, size + kPieceOverhead) + c * kPartAdd;
        if (time < least) {
          least = time;
          choice = users | c << 16;
        }
      }
      // The least time of all, ties to the fewest cuts (non-negative floats order like their bits).
      auto lowest = [&](unsigned time) {
        const unsigned t = __reduce_min_sync(0xffffffffu, time);
        choice = (int)__reduce_min_sync(0xffffffffu, time == t ? (unsigned)choice : UINT_MAX);
        return t;
      };
      unsigned t = lowest(__float_as_uint(least));
      if ((tid & 31) == 0) s_choice[tid >> 5] = make_int2((int)t, choice);
      __syncthreads();
      const int2 other = s_choice[min(tid & 31, kSchedWarps - 1)];
      choice = other.y;
      lowest((unsigned)other.x);
    }
    cut_users = choice & 0xffff;
    if (cut_users > 0) q = cdiv(top, choice >> 16);
  }
  const int cut_blocks = cut_users > 0 ? s_start[cut_users] : 0;  // they are the first ones
  const int whole = items - cut_blocks * a.H;
  if (cut_users > 0) {
    // Queue places: user, head, part, block.  Every item of a user is cut alike; the places of parts
    // that a short item does not have stay empty.
    const int mine = tid < cut_users ? (s_start[tid + 1] - s_start[tid]) * a.H * cdiv(s_cost[tid], q) : 0;
    const int first = paged_scan(mine, scratch, &cut_places) - mine;
    if (tid < cut_users) s_tiles[tid] = first;
    __syncthreads();
#pragma unroll 1
    for (int x = tid; x < cut_blocks * a.H; x += kSchedThreads) {
      const int h = x / cut_blocks;
      int b, blk, cost;
      block_of(x - h * cut_blocks, b, blk, cost);
      PagedPiece p = piece_of(b, blk, cost);
      p.h = h;
      const int parts = cdiv(s_cost[b], q);
      p.pitch = s_start[b + 1] - s_start[b];
      p.parts = min(parts, cost);
      const int at = s_tiles[b] + h * parts * p.pitch + blk;
#pragma unroll 1
      for (p.part = 0; p.part < parts; ++p.part) {
        p.tile0 = p.part < p.parts ? cost * p.part / p.parts : 0;
        p.tiles = p.part < p.parts ? cost * (p.part + 1) / p.parts - p.tile0 : 0;
        put(whole + at + p.part * p.pitch, p);
      }
      reinterpret_cast<int4*>(a.plan.done)[at] = make_int4(0, 0, 0, 0);
    }
  }
  if (tid == 0) *reinterpret_cast<int4*>(a.plan.header) = make_int4(0, whole + cut_places, whole, 0);
  if (whole == 0) return;

  // Whole items: a counting sort of the blocks by (wave, non-increasing cost).  Waves are those the batch
  // reaches, or fewer that hold more; costs are rounded to bins that fit the key space.
  const int wave_tiles = max(1, a.wave_rows / kTileRows);
  int shift = 0;
  while ((top >> shift) >= kMaxCostBins / 2) ++shift;
  const int bins = (top >> shift) + 1;
  const int waves = min(few_users ? (int)(carry >> 32) / wave_tiles + 1 : 16, kMaxCostBins / bins);
  const int nkeys = bins * waves;
  auto key_of = [&](int b, int cost) {
    const int wave = few_users ? min(s_tiles[b] / wave_tiles, waves - 1) : (int)((int64_t)b * waves / a.B);
    return wave * bins + ((top - cost) >> shift);
  };
  // Lanes with the same key add to it together: equal costs are the rule.
  auto claim = [&](int key, int& rank) {
    const unsigned same = __match_any_sync(0xffffffffu, key);
    rank = __popc(same & ((1u << (tid & 31)) - 1u));
    const int leader = __ffs(same) - 1;
    int at = 0;
    if (key >= 0 && rank == 0) at = atomicAdd(&hist[key], __popc(same) * a.H);
    return __shfl_sync(0xffffffffu, at, leader);
  };
  const int rounds = cdiv(nblocks - cut_blocks, kSchedThreads);
#pragma unroll 1
  for (int k = 0; k < rounds; ++k) {
    int b, blk, cost, rank, key = -1;
    if (cut_blocks + k * kSchedThreads + tid < nblocks) {
      block_of(cut_blocks + k * kSchedThreads + tid, b, blk, cost);
      key = key_of(b, cost);
    }
    claim(key, rank);
  }
  __syncthreads();
  const int per = cdiv(nkeys, kSchedThreads);
  int part = 0, total;
#pragma unroll 1
  for (int k = 0; k < per; ++k)
    if (tid * per + k < nkeys) part += hist[tid * per + k];
  int run = paged_scan(part, scratch, &total) - part;
#pragma unroll 1
  for (int k = 0; k < per; ++k) {
    const int key = tid * per + k;
    if (key < nkeys) {
      const int n = hist[key];
      hist[key] = run;
      run += n;
    }
  }
  __syncthreads();
#pragma unroll 1
  for (int k = 0; k < rounds; ++k) {
    const bool there = cut_blocks + k * kSchedThreads + tid < nblocks;
    int b, blk, cost, rank, key = -1;
    if (there) {
      block_of(cut_blocks + k * kSchedThreads + tid, b, blk, cost);
      key = key_of(b, cost);
    }
    const int at = claim(key, rank);
    if (!there) continue;
    PagedPiece p = piece_of(b, blk, cost);
#pragma unroll 1
    for (p.h = 0; p.h < a.H; ++p.h) put(at + rank * a.H + p.h, p);
  }
}

}  // namespace hstu
