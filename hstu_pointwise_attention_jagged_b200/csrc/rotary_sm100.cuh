// rotary_sm100.cuh — position rotation of token rows, written to packed or strided rows (hstu_rotary)
// or, for K and V, to their places in a paged cache (hstu_paged_append).
//
// A pair (x, y) of a head turns by t = pos * freq: (x cos t - y sin t, x sin t + y cos t).  One
// cos/sin pair serves every head of Q and of K, so a block of R rows first forms its R x pairs table
// in shared memory and then streams its rows through it.  What bounds the kernel is the rows' bytes, read
// and written once (4 bytes an element): the first batch of 32-byte units is loaded before the
// table is formed, so the row traffic covers the angles' arithmetic.
//
// Angles.  pos is up to 2^31 (Unix times), where pos * freq in fp32 has no correct digit left.  The
// angle is formed in turns, pos * (freq / 2 pi), in fp64; only its fraction, exact to 2^-53 of the
// whole, is rounded to fp32 and goes to sincospif.
#pragma once

#include <climits>
#include <cstdint>
#include <cuda_bf16.h>

#include "hstu_fwd_sm100.cuh"
#include "paged_cache.cuh"

namespace hstu {

constexpr int kRotThreads = 256;
constexpr int kRotBatch = 4;        // 32-byte units a thread has in flight
constexpr int kRotMaxRows = 16;     // rows of a block
constexpr int kRotMaxPairs = 64;
constexpr int kRotScanUsers = 1024; // batches up to this size: each block scans the offsets for its rows' users

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
  int32_t tensors, rows, rows_per_block, H;
  int32_t head_shift;   // log2(d / 16): 32-byte units of a head
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

template <bool kPaged>
__global__ void __launch_bounds__(kRotThreads) rotary_kernel(const RotArgs p) {
  // (cos, sin) of row r, pair 8 u + 2 j + e at float2 index ((r * 4 + j) * (pairs / 8) + u) * 2 + e, so
  // that neighbouring units read neighbouring float4.
  __shared__ float4 s_cs[kRotMaxRows * kRotMaxPairs / 2];
  __shared__ int64_t s_dst[kRotMaxRows];  // element offset of the row in the cache, -1: not written
  __shared__ int32_t s_place[kRotMaxRows], s_user[kRotMaxRows];
  const int tid = threadIdx.x;
  const int row0 = blockIdx.x * p.rows_per_block;
  const int nrows = min(p.rows_per_block, p.rows - row0);
  const int pairs = p.pairs;
  const uint32_t head_units = 1u << p.head_shift;
  const uint32_t units = (uint32_t)nrows * p.tensors * p.H * head_units;

  // Unit x of the block: its row, tensor and the columns of its two vectors.
  struct Place {
    int r, t;
    int c0, c1;
    bool turn;
    int part;
  };
  auto place_of = [&](uint32_t x) {
    Place u;
    u.part = (int)(x & (head_units - 1));
    const uint32_t y = x >> p.head_shift;
    const uint32_t rt = y / (uint32_t)p.H;
    const int h = (int)(y - rt * p.H);
    u.r = (int)(rt / (uint32_t)p.tensors);
    u.t = (int)(rt - (uint32_t)u.r * p.tensors);
    u.turn = p.t[u.t].rotated && u.part * 8 < pairs;
    const int head0 = h << (p.head_shift + 4);
    const bool split = u.turn && !p.interleaved;
    u.c0 = head0 + (split ? u.part * 8 : u.part * 16);
    u.c1 = split ? u.c0 + pairs : u.c0 + 8;
    return u;
  };
  RotUnit held[kRotBatch];
  auto load_batch = [&](uint32_t x0) {
#pragma unroll
    for (int i = 0; i < kRotBatch; ++i) {
      const uint32_t x = x0 + i * kRotThreads;
      if (x < units) {
        const Place u = place_of(x);
        const __nv_bfloat16* src = p.t[u.t].src + (int64_t)(row0 + u.r) * p.t[u.t].src_ld;
        held[i].a = __ldcs(reinterpret_cast<const uint4*>(src + u.c0));
        held[i].b = __ldcs(reinterpret_cast<const uint4*>(src + u.c1));
      }
    }
  };
  load_batch(tid);

  if constexpr (kPaged) {
    // Whose rows these are.  Up to kRotScanUsers users every block looks at all offsets, which costs one
    // round of coalesced loads; beyond that each row searches for itself.
    if (tid < kRotMaxRows) s_user[tid] = INT_MAX;
    __syncthreads();
    if (p.B <= kRotScanUsers) {
      for (int b = tid; b < p.B; b += kRotThreads) {
        const int o0 = p.q_offsets[b], o1 = p.q_offsets[b + 1];
        const int hi = min(o1, row0 + nrows);
        for (int r = max(o0, row0); r < hi; ++r) atomicMin(&s_user[r - row0], b);
      }
    } else if (tid < nrows) {
      int lo = 0, hi = p.B;
      while (hi - lo > 1) {
        const int mid = lo + (hi - lo) / 2;
        if (p.q_offsets[mid] <= row0 + tid) lo = mid; else hi = mid;
      }
      if (p.q_offsets[lo] <= row0 + tid && row0 + tid < p.q_offsets[lo + 1]) s_user[tid] = lo;
    }
    if (blockIdx.x == 0) {
      bool bad = tid == 0 && (p.q_offsets[0] != 0 || p.q_offsets[p.B] != p.rows);
      for (int b = tid; b < p.B; b += kRotThreads)
        bad |= !paged_user(p.cache, p.q_offsets, p.kv_len, nullptr, b, p.rows, INT_MAX, -1).ok;
      if (bad) atomicOr(p.err, kErrBadOffsets);
    }
    __syncthreads();
    if (tid < nrows) {
      int64_t dst = -1;
      int place = -1;
      const int b = s_user[tid];
      if (b != INT_MAX) {
        const PagedUser u = paged_user(p.cache, p.q_offsets, p.kv_len, nullptr, b, p.rows, INT_MAX, -1);
        if (u.ok) {
          place = u.L - u.n + (row0 + tid - u.q0);
          const int page = p.cache.table[b * p.cache.table_ld + (place >> p.cache.page_shift)];
          if (page >= 0 && page < p.cache.num_pages)
            dst = page * p.cache.page_stride + (place & ((1 << p.cache.page_shift) - 1)) * p.cache.row_stride;
          else
            atomicOr(p.err, kErrBadOffsets);
        }
      }
      s_dst[tid] = dst;
      s_place[tid] = place;
    }
    __syncthreads();
  }

  for (int x = tid; x < nrows * pairs; x += kRotThreads) {
    const int r = x / pairs, i = x - r * pairs;
    const int axis = (p.axes > 1 && i >= p.section_end[0]) + (p.axes > 2 && i >= p.section_end[1]) +
                     (p.axes > 3 && i >= p.section_end[2]);
    int pos;
    if (kPaged && p.positions == nullptr) pos = s_place[r];
    else pos = p.positions[axis * p.positions_ld + row0 + r];
    constexpr double kInv2Pi = 0.15915494309189533577;
    const double turns = pos * (p.freqs[i] * kInv2Pi);
    float sn, cs;
    sincospif(2.0f * (float)(turns - rint(turns)), &sn, &cs);
    reinterpret_cast<float2*>(s_cs)[((r * 4 + ((i >> 1) & 3)) * (pairs >> 3) + (i >> 3)) * 2 + (i & 1)] =
        make_float2(cs, p.sign * sn);
  }
  __syncthreads();

  const int64_t cache_head = p.cache.head_stride;
  for (uint32_t x0 = tid; x0 < units; x0 += kRotBatch * kRotThreads) {
    if (x0 != (uint32_t)tid) load_batch(x0);
#pragma unroll
    for (int i = 0; i < kRotBatch; ++i) {
      const uint32_t x = x0 + i * kRotThreads;
      if (x >= units) break;
      const Place u = place_of(x);
      if (u.turn) {
        float4 cs[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) cs[j] = s_cs[(u.r * 4 + j) * (pairs >> 3) + u.part];
        turn_unit(held[i], cs, p.interleaved);
      }
      const RotTensor& t = p.t[u.t];
      __nv_bfloat16 *d0, *d1;
      if (kPaged && t.target != kToRows) {
        if (s_dst[u.r] < 0) continue;
        const int d_mask = (16 << p.head_shift) - 1;
        __nv_bfloat16* base = (t.target == kToCacheK ? p.cache.k : p.cache.v) + s_dst[u.r] +
                              (u.c0 >> (p.head_shift + 4)) * cache_head;
        d0 = base + (u.c0 & d_mask);
        d1 = base + (u.c1 & d_mask);
      } else {
        if (kPaged && s_place[u.r] < 0) continue;
        __nv_bfloat16* base = t.dst + (int64_t)(row0 + u.r) * t.dst_ld;
        d0 = base + u.c0;
        d1 = base + u.c1;
      }
      *reinterpret_cast<uint4*>(d0) = held[i].a;
      *reinterpret_cast<uint4*>(d1) = held[i].b;
    }
  }
}

}  // namespace hstu
