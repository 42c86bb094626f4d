// schedule.cuh — tile geometry of the target-aware mask and the parts that the work plans share.
//
// Mask (DLRMv3 review, section "model selection": history encoded once and shared by every
// candidate; infolabhq.com multi-stage page: the user side never depends on a candidate, and
// target-aware attention weighs the history against each candidate):
//   query at position i of a segment with U history tokens may see key j iff
//     i <  U : j <= i                 (history token, causal over the history)
//     i >= U : j <  U  or  j == i     (candidate: all history, then itself)
// The keys visible to a block of queries at positions [p0, p1) are therefore
//     [0, p1)                         if p1 <= U
//     [0, U)  +  [max(p0, U), p1)     otherwise,
// i.e. at most two runs of 128-key tiles.  Tiles outside them are never enumerated.
#pragma once

#include <cstdint>

namespace hstu {

constexpr int kTileRows = 128;  // query rows per half / keys per key tile
constexpr int kItemRows = 128;  // query rows per work item: one query tile

__host__ __device__ __forceinline__ int cdiv(int a, int b) { return (a + b - 1) / b; }

// Key tiles [0, e1) followed by [s2, e2), with s2 >= e1 (an empty second run has s2 == e2).
struct TileRange {
  int e1, s2, e2;
};

// kKeys: keys of a tile.
template <int kKeys = kTileRows>
__host__ __device__ __forceinline__ TileRange key_tiles(int p0, int p1, int U) {
  TileRange r{0, 0, 0};
  if (p1 <= p0) return r;
  if (p1 <= U) {
    r.e1 = cdiv(p1, kKeys);
    r.s2 = r.e2 = r.e1;
    return r;
  }
  r.e1 = cdiv(U, kKeys);
  const int s = (p0 > U ? p0 : U) / kKeys;
  const int e = cdiv(p1, kKeys);
  if (s <= r.e1) {
    r.e1 = (e > r.e1) ? e : r.e1;
    r.s2 = r.e2 = r.e1;
  } else {
    r.s2 = s;
    r.e2 = e;
  }
  return r;
}

__host__ __device__ __forceinline__ int tile_count(const TileRange& r) { return r.e1 + (r.e2 - r.s2); }
__host__ __device__ __forceinline__ int tile_at(const TileRange& r, int idx) {
  return idx < r.e1 ? idx : r.s2 + (idx - r.e1);
}
__host__ __device__ __forceinline__ bool tile_in(const TileRange& r, int t) {
  return t < r.e1 || (t >= r.s2 && t < r.e2);
}

// Score tiles computed by one work item: query rows [128*blk, 128*blk + nrows) at positions
// pos0.. of a segment with U history tokens.
__host__ __device__ __forceinline__ int item_cost(int pos0, int nrows, int U) {
  return nrows > 0 ? tile_count(key_tiles(pos0, pos0 + nrows, U)) : 0;
}

constexpr unsigned kErrBadOffsets = 1u;
constexpr unsigned kErrTimeout = 2u;

constexpr int kSchedThreads = 256;
constexpr int kSchedWarps = kSchedThreads / 32;
constexpr int kMaxCostBins = 4096;
constexpr int kCachedUsers = 256;  // batches up to this many users keep per-user values in shared memory

// Score tiles of a 128-row item at most: ceil(L/128) + 1.
inline int cost_bound(int32_t max_seq_len) { return max_seq_len / kTileRows + 2; }

// Cost bins a plan needs: twice the room that the costs take.
inline int cost_bins(int32_t max_seq_len) {
  const int64_t n = 2 * (static_cast<int64_t>(cost_bound(max_seq_len)) + 1) + 1;
  return static_cast<int>(n < kMaxCostBins ? n : kMaxCostBins);
}

// Waves a plan's keys need: those the batch's rows can reach, no more than the key space holds (the
// plan kernels clear and scan waves x cost bins keys).
inline int plan_waves(int64_t rows, int32_t wave_rows, int32_t nbins) {
  const int64_t need = rows > 0 ? (rows + wave_rows - 1) / wave_rows : 1;
  const int64_t fit = nbins > 0 ? kMaxCostBins / nbins : 1;
  const int64_t n = need < fit ? need : fit;
  return static_cast<int>(n > 0 ? n : 1);
}

// Rows of a wave: users whose K and V (sized for d = 128: 512 bytes per row and head) take about a
// quarter of the 126 MB L2.
inline int32_t plan_wave_rows(int32_t H) {
  const int64_t n = (32ll << 20) / (512ll * H);
  return static_cast<int32_t>(n > 0 ? n : 1);
}

// Inclusive block-wide prefix sums of two values per thread (kSchedThreads threads); also
// returns the block totals.  `scratch` holds 2 x 32 values.
__device__ __forceinline__ void block_inclusive_scan2(long long& a, long long& b, long long (*scratch)[32],
                                                      long long& total_a, long long& total_b) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long na = __shfl_up_sync(0xffffffffu, a, o);
    const long long nb = __shfl_up_sync(0xffffffffu, b, o);
    if (lane >= o) {
      a += na;
      b += nb;
    }
  }
  if (lane == 31) {
    scratch[0][warp] = a;
    scratch[1][warp] = b;
  }
  __syncthreads();
  if (warp == 0) {
    long long wa = lane < kSchedWarps ? scratch[0][lane] : 0, wb = lane < kSchedWarps ? scratch[1][lane] : 0;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long na = __shfl_up_sync(0xffffffffu, wa, o);
      const long long nb = __shfl_up_sync(0xffffffffu, wb, o);
      if (lane >= o) {
        wa += na;
        wb += nb;
      }
    }
    scratch[0][lane] = wa;
    scratch[1][lane] = wb;
  }
  __syncthreads();
  if (warp > 0) {
    a += scratch[0][warp - 1];
    b += scratch[1][warp - 1];
  }
  total_a = scratch[0][kSchedWarps - 1];
  total_b = scratch[1][kSchedWarps - 1];
  __syncthreads();
}

// Inclusive block-wide prefix sum of one value per thread (kSchedThreads threads); also
// returns the block total.  `scratch` holds 32 values.
__device__ __forceinline__ long long block_inclusive_scan(long long v, long long* scratch,
                                                          long long* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    long long n = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += n;
  }
  if (lane == 31) scratch[warp] = v;
  __syncthreads();
  if (warp == 0) {
    long long w = lane < kSchedWarps ? scratch[lane] : 0;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      long long n = __shfl_up_sync(0xffffffffu, w, o);
      if (lane >= o) w += n;
    }
    scratch[lane] = w;
  }
  __syncthreads();
  if (warp > 0) v += scratch[warp - 1];
  *total = scratch[kSchedWarps - 1];
  __syncthreads();
  return v;
}

// User owning block g: the last b with block_start[b] <= g (users without blocks share a start).
// block_start may live in shared or global memory.
__device__ __forceinline__ int owner_of(const int32_t* block_start, int B, int g) {
  int lo = 0, hi = B;  // block_start[lo] <= g < block_start[hi]
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (block_start[mid] <= g) lo = mid; else hi = mid;
  }
  return lo;
}

}  // namespace hstu
