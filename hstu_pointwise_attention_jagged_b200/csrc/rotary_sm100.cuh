// rotary_sm100.cuh — position rotation of token rows, written to packed or strided rows (hstu_rotary)
// or, for K and V, to their places in a paged cache (hstu_paged_append).
//
// A pair (x, y) of a head turns by t = pos * freq: (x cos t - y sin t, x sin t + y cos t).  One
// cos/sin pair serves every head of Q and of K, so a block of rows first forms its rows x pairs table
// in shared memory and then streams its rows through it.  What bounds the kernel is the rows' bytes, read
// and written once (4 bytes an element), if the instructions for a 32-byte unit stay few: a thread
// keeps one place within the row (tensor, head, columns), decoded once, and steps through rows.  Its
// first units are loaded before the table is formed, so their latency covers the angles' arithmetic
// and the look-ups in offsets and page table.
//
// Angles.  pos is up to 2^31 (Unix times), where pos * freq in fp32 has no correct digit left.  They are
// formed in turns, in 64-bit fixed point: freq / 2 pi modulo one turn is a whole number of 2^-64 turns,
// its product with pos wraps modulo one turn by itself, and the upper half of it goes to sincospif.
#pragma once

#include <climits>
#include <cstdint>
#include <cuda_bf16.h>

#include "hstu_fwd_sm100.cuh"
#include "paged_cache.cuh"

namespace hstu {

constexpr int kRotThreads = 256;    // at most
// Units a thread has in flight, and how often over (measured at 2 x 2, 4 x 1, 2 x 4, 3 x 2 and 1 x 4: rotation of
// 32768 x 512 Q and K in 23.7, 26.3, 24.0, 23.8 and 25.6 us, streaming append 42.1, 46.1, 45.2, 42.2 and 44.1).
constexpr int kRotBatch = 2, kRotPasses = 2;
constexpr int kRotSideRows = 16;    // rows side by side at most
constexpr int kRotMaxRows = kRotSideRows * kRotBatch * kRotPasses;  // rows of a block
constexpr int kRotMaxPairs = 64;

enum RotTarget : int32_t { kToRows = 0, kToCacheK = 1, kToCacheV = 2 };

struct RotTensor {
  const __nv_bfloat16* src;
  int64_t src_ld;
  __nv_bfloat16* dst;  // kToRows
  int64_t dst_ld;
  int32_t target;
  int32_t rotated;
};

struct RotArgs {
  RotTensor t[3];
  int32_t tensors, rows, H;
  int32_t head_shift;   // log2(d / 16): 32-byte units of a head
  // A block takes `block_rows` rows, `side_rows` of them side by side: thread x has place x % row_units of
  // rows x / row_units + k * side_rows (one row at a time, several places, when a row has more units than
  // the block has threads).
  int32_t row_units, side_rows, block_rows;
  // rotation; pairs = 0 for plain copies
  const double* freqs;
  const int32_t* positions;  // null: the row's place in the cache
  int64_t positions_ld;
  int32_t pairs, axes, section_end[3];  // pair i belongs to the first axis a with i < section_end[a]
  int32_t interleaved;
  float sign;
  // paged targets
  PagedView cache;
  const int32_t* q_offsets;
  const int32_t* kv_len;
  int32_t B;
  unsigned* err;
};

// A unit: two 16-byte vectors of one head, eight pairs where the head's columns turn.
struct RotUnit {
  uint4 a, b;
};

// Turns the unit's pairs; cs[j] = (cos, sin) of pairs 2j and 2j + 1.
__device__ __forceinline__ void turn_unit(RotUnit& u, const float4 (&cs)[4], bool interleaved) {
  uint32_t wa[4] = {u.a.x, u.a.y, u.a.z, u.a.w}, wb[4] = {u.b.x, u.b.y, u.b.z, u.b.w};
  auto lo = [](uint32_t w) { return __uint_as_float(w << 16); };
  auto hi = [](uint32_t w) { return __uint_as_float(w & 0xffff0000u); };
  if (interleaved) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      // word j of `a` is pair j, word j of `b` pair 4 + j
      const float4 ca = cs[j >> 1], cb = cs[2 + (j >> 1)];
      const float c0 = (j & 1) ? ca.z : ca.x, s0 = (j & 1) ? ca.w : ca.y;
      const float c1 = (j & 1) ? cb.z : cb.x, s1 = (j & 1) ? cb.w : cb.y;
      const float x0 = lo(wa[j]), y0 = hi(wa[j]), x1 = lo(wb[j]), y1 = hi(wb[j]);
      wa[j] = pack_bf16x2(x0 * c0 - y0 * s0, x0 * s0 + y0 * c0);
      wb[j] = pack_bf16x2(x1 * c1 - y1 * s1, x1 * s1 + y1 * c1);
    }
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float x0 = lo(wa[j]), x1 = hi(wa[j]), y0 = lo(wb[j]), y1 = hi(wb[j]);
      wa[j] = pack_bf16x2(x0 * cs[j].x - y0 * cs[j].y, x1 * cs[j].z - y1 * cs[j].w);
      wb[j] = pack_bf16x2(x0 * cs[j].y + y0 * cs[j].x, x1 * cs[j].w + y1 * cs[j].z);
    }
  }
  u.a = make_uint4(wa[0], wa[1], wa[2], wa[3]);
  u.b = make_uint4(wb[0], wb[1], wb[2], wb[3]);
}

// freq (radians) as 2^-64 turns, modulo one turn.  The nearest whole turn is taken off, which is exact for both
// signs: with the one below, a small negative freq would be rounded to 2^-54 turns, 7e-7 radians at a far position.
__device__ __forceinline__ uint64_t turns_of(double freq) {
  const double t = freq * 0.15915494309189533577;  // 1 / 2 pi
  return (uint64_t)__double2ll_rz((t - rint(t)) * 0x1p64);  // half a turn saturates, 2^-64 turns short of it
}

template <bool kPaged>
__global__ void __launch_bounds__(kRotThreads, 4) rotary_kernel(const RotArgs p) {
  // (cos, sin) of row r, pair 8 u + 2 j + e at float2 index ((r * 4 + j) * (pairs / 8) + u) * 2 + e, so
  // that neighbouring units read neighbouring float4.
  extern __shared__ float4 s_cs[];
  __shared__ int64_t s_dst[kRotMaxRows];    // element offset of the row in the cache, -1: not written
  __shared__ int32_t s_place[kRotMaxRows];  // the row's place in its user's cache, -1: no user's row
  const int tid = threadIdx.x, threads = blockDim.x;
  const int row0 = blockIdx.x * p.block_rows;
  const int nrows = min(p.block_rows, p.rows - row0);
  const int pairs = p.pairs;
  const int per_pass = p.side_rows * p.row_units;  // threads that take part

  // Unit place x of a row: its tensor and the columns of its two vectors.
  struct Place {
    int t, h, c0, c1, part;  // c0, c1: within the head
    bool turn;
  };
  auto place_of = [&](int x) {
    Place u;
    u.part = x & ((1 << p.head_shift) - 1);
    const int y = x >> p.head_shift;
    u.t = y / p.H;
    u.h = y - u.t * p.H;
    u.turn = p.t[u.t].rotated && u.part * 8 < pairs;
    const bool split = u.turn && !p.interleaved;
    u.c0 = split ? u.part * 8 : u.part * 16;
    u.c1 = split ? u.c0 + pairs : u.c0 + 8;
    return u;
  };
  const int side = tid / p.row_units;  // 0 when a row has more units than the block has threads
  RotUnit held[kRotBatch];
  const __nv_bfloat16* src = nullptr;
  int64_t src_step = 0;
  auto aim = [&](const Place& u) {
    const RotTensor& t = p.t[u.t];
    src = t.src + (int64_t)(row0 + side) * t.src_ld + (u.h << (p.head_shift + 4));
    src_step = p.side_rows * t.src_ld;
  };
  auto load_batch = [&](const Place& u, int r) {
    const __nv_bfloat16* from = src;
#pragma unroll
    for (int i = 0; i < kRotBatch; ++i) {
      if (r + i * p.side_rows < nrows) {
        held[i].a = __ldcs(reinterpret_cast<const uint4*>(from + u.c0));
        held[i].b = __ldcs(reinterpret_cast<const uint4*>(from + u.c1));
      }
      from += src_step;
    }
    src = from;
  };
  const bool active = tid < per_pass || per_pass > threads;
  int x = side == 0 ? tid : tid - side * p.row_units;
  Place u = place_of(x < p.row_units ? x : 0);
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (active) {
    aim(u);
    load_batch(u, side);
  }

  auto angles = [&] {
    // Thread -> pair tid % pairs of rows tid / pairs + k * (threads / pairs).
    const int i = tid % pairs, step = threads / pairs;
    if (tid >= step * pairs) return;
    const int axis = (p.axes > 1 && i >= p.section_end[0]) + (p.axes > 2 && i >= p.section_end[1]) +
                     (p.axes > 3 && i >= p.section_end[2]);
    const uint64_t turns = turns_of(p.freqs[i]);
    const int32_t* pos = p.positions ? p.positions + axis * p.positions_ld + row0 : nullptr;
    float2* to = reinterpret_cast<float2*>(s_cs) + (((i >> 1) & 3) * (pairs >> 3) + (i >> 3)) * 2 + (i & 1);
    for (int r = tid / pairs; r < nrows; r += step) {
      const int at = pos ? pos[r] : s_place[r];
      const int part = (int)(uint32_t)(((uint64_t)(int64_t)at * turns) >> 32);  // 2^-32 turns, signed
      float sn, cs;
      sincospif((float)part * 0x1p-31f, &sn, &cs);
      to[r * pairs] = make_float2(cs, p.sign * sn);
    }
  };

  if constexpr (kPaged) {
    // Whose row this is and where it goes: a thread for each row, kRotMaxRows at most and no more than there
    // are threads.  The search's loads hit L1 after the SM's first block.
    if (tid < nrows) {
      const int row = row0 + tid;
      int lo = 0, hi = p.B;
      while (hi - lo > 1) {
        const int mid = lo + (hi - lo) / 2;
        if (p.q_offsets[mid] <= row) lo = mid; else hi = mid;
      }
      const PagedUser v = paged_user(p.cache, p.q_offsets, p.kv_len, nullptr, lo, p.rows, INT_MAX, -1);
      int64_t dst = -1;
      int place = -1;
      if (v.ok && v.q0 <= row && row < v.q0 + v.n) {
        place = v.L - v.n + (row - v.q0);
        const int page = p.cache.table[lo * p.cache.table_ld + (place >> p.cache.page_shift)];
        if (page >= 0 && page < p.cache.num_pages)
          dst = page * p.cache.page_stride + (place & ((1 << p.cache.page_shift) - 1)) * p.cache.row_stride;
        else
          atomicOr(p.err, kErrBadOffsets);
      }
      s_dst[tid] = dst;
      s_place[tid] = place;
    }
    if (blockIdx.x == 0) {
      bool bad = tid == 0 && (p.q_offsets[0] != 0 || p.q_offsets[p.B] != p.rows);
      for (int b = tid; b < p.B; b += threads)
        bad |= !paged_user(p.cache, p.q_offsets, p.kv_len, nullptr, b, p.rows, INT_MAX, -1).ok;
      if (bad) atomicOr(p.err, kErrBadOffsets);
    }
    if (pairs > 0 && p.positions == nullptr) __syncthreads();  // the angles are of the places
  }
  if (pairs > 0) angles();
  __syncthreads();
  if (!active) return;

  while (true) {
    const RotTensor& t = p.t[u.t];
    const bool cached = kPaged && t.target != kToRows;
    __nv_bfloat16* base = cached ? (t.target == kToCacheK ? p.cache.k : p.cache.v) + u.h * p.cache.head_stride
                                 : t.dst + (int64_t)row0 * t.dst_ld + (u.h << (p.head_shift + 4));
    for (int r0 = side; r0 < nrows; r0 += kRotBatch * p.side_rows) {
      if (r0 != side) load_batch(u, r0);
#pragma unroll
      for (int i = 0; i < kRotBatch; ++i) {
        const int r = r0 + i * p.side_rows;
        if (r >= nrows) break;
        if (u.turn) {
          float4 cs[4];
#pragma unroll
          for (int j = 0; j < 4; ++j) cs[j] = s_cs[(r * 4 + j) * (pairs >> 3) + u.part];
          turn_unit(held[i], cs, p.interleaved);
        }
        int64_t to;
        if (cached) {
          to = s_dst[r];
          if (to < 0) continue;
        } else {
          if (kPaged && s_place[r] < 0) continue;
          to = r * t.dst_ld;
        }
        *reinterpret_cast<uint4*>(base + to + u.c0) = held[i].a;
        *reinterpret_cast<uint4*>(base + to + u.c1) = held[i].b;
      }
    }
    x += threads;
    if (per_pass <= threads || x >= p.row_units) break;
    u = place_of(x);
    aim(u);
    load_batch(u, side);
  }
}

}  // namespace hstu
