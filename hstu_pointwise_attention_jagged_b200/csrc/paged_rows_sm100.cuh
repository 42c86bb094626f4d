// paged_rows_sm100.cuh — target-aware SiLU attention of a few new rows a user over the paged cache.
//
// With up to 16 query rows a user the work is a pass over the user's cached K and V: 2 * L * d * 2
// bytes a head for at most 16 * L * d * 4 flops, so the bound is DRAM and the tensor cores only have
// to stay out of the way.  A 128-row tcgen05 tile would be empty but for those rows; the warp-level
// m16n8k16 product takes exactly 16 rows from shared memory and keeps S, P and O in registers.
//
// A CTA streams key tiles through kRowsStages buffers of cp.async copies; its four warps take a
// quarter of each tile's keys, each with its own O.  A tile is 16 KB of K and 16 KB of V: 64, 128 or 256
// keys for d = 128, 64, 32, so that every thread copies 8 consecutive rows of one 16-byte column; 8
// aligned rows never cross a page, and the table is read a tile ahead.  Rows past the user's length
// are filled with zeros, whatever the page holds there.  (A producer warp with TMA copies of the pages was
// slower: 5.1 against 3.0 us for the smallest calls, 1.26 times the time a tile for one CTA.)
//
// SiLU attention has no softmax statistics, so an item's (user's and head's) key tiles can be shared
// out freely and the partial O's simply add up.  Two kernels do that differently:
//   paged_rows_kernel      one cluster of CTAs for each item; the partial O's are added over distributed
//                          shared memory, in rank order.  One launch and no workspace: for calls whose
//                          time is latency, and for batches of so many items that each needs one CTA.
//                          More than 16 rows a user become several items while the call stays short.
//   paged_rows_run_kernel  the tiles of all items, in item order, dealt out in equal runs to two CTAs for
//                          each SM; parts of items go to a workspace and paged_rows_sum_kernel adds them in
//                          order.  Ragged lengths and any number of items load every SM alike.
// No sum depends on timing.
#pragma once

#include <cstdint>
#include <cuda_bf16.h>

#include "hstu_fwd_sm100.cuh"
#include "paged_cache.cuh"
#include "schedule.cuh"
#include "sm100_ptx.cuh"

namespace hstu {

constexpr int kRowsThreads = 128;
constexpr int kRowsBlock = 16;        // query rows of a CTA
constexpr int kRowsStages = 3;
constexpr int kRowsMaxSplit = 16;     // CTAs of a cluster
constexpr int kRowsClusterTiles = 16; // tiles of a CTA of a cluster at most
constexpr int kRowsBlocksTiles = 12;  // with several blocks a user: tiles in all, for each CTA the GPU holds

template <int D>
struct RowsCfg {
  static constexpr int kRowBytes = D * 2;
  static constexpr int kChunks = kRowBytes / 16;        // 16-byte columns of a row
  static constexpr int kKeys = 64 * 128 / D;            // keys of a tile
  static constexpr int kWarpKeys = kKeys / 4;
  static constexpr int kTileBytes = kKeys * kRowBytes;  // 16 KB
  static constexpr int kStageBytes = 2 * kTileBytes;    // K, then V
  static constexpr int kSmemBytes = kRowsStages * kStageBytes;
  static_assert(4 * kRowsBlock * (D + 8) * 4 <= kSmemBytes, "the warps' sums reuse the tiles");
  static_assert(4 * kRowsBlock * D * 4 <= kStageBytes, "and fit one stage unpadded");
  // Offset of 16-byte column c of row r: eight consecutive rows hit eight 16-byte bank groups.
  __device__ static __forceinline__ uint32_t at(int r, int c) {
    return r * kRowBytes + ((D == 32 ? (c ^ ((r >> 1) & 3)) : (c ^ (r & 7))) << 4);
  }
};

struct RowsArgs {
  const __nv_bfloat16* q;
  int64_t q_ld;
  __nv_bfloat16* out;
  int64_t out_ld;
  PagedView cache;
  const int32_t* q_offsets;
  const int32_t* kv_len;
  const int32_t* num_targets;  // may be null
  int32_t B, H, total_new, max_new, max_kv;
  int32_t blocks;  // 16-row blocks of a user's rows, at most; an item is one of them
  float half_alpha, inv_n;
  unsigned* err;
};

namespace ptx {

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, uint32_t bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int kLeft>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(kLeft) : "memory");
}
__device__ __forceinline__ void ldmatrix4(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldmatrix4_trans(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
// The transpose of an 8 x 8 matrix of 16-bit values held as one ldmatrix fragment.
__device__ __forceinline__ uint32_t transpose_8x8(uint32_t a) {
  uint32_t d;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(a));
  return d;
}
// c += a (16 x 16) * b (16 x 8), bf16 in, fp32 sums.
__device__ __forceinline__ void mma_16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// Shared memory of another CTA of the cluster (address from mapa_shared).
__device__ __forceinline__ float4 ld_cluster_v4(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(addr)
               : "memory");
  return v;
}

}  // namespace ptx

// ---------------------------------------------------------------------------------------------
// Parts of both kernels
// ---------------------------------------------------------------------------------------------
// Where this thread copies from and to: 16-byte column tid % kChunks of rows 8 (tid / kChunks) .. + 8.
template <int D>
struct RowsCopy {
  using Cfg = RowsCfg<D>;
  int col, rbase;
  __device__ __forceinline__ RowsCopy() : col(threadIdx.x % Cfg::kChunks), rbase(threadIdx.x / Cfg::kChunks * 8) {}

  // Table entry of this thread's rows of the tile at key0 of user b (length L).
  __device__ __forceinline__ int look_up(const PagedView& c, int b, int L, int key0) const {
    return key0 + rbase < L ? c.table[b * c.table_ld + ((key0 + rbase) >> c.page_shift)] : 0;
  }

  // Keys [key0, key0 + kKeys) of head h into the buffer at shared address `dst`; page: from look_up.
  __device__ __forceinline__ void issue(const PagedView& c, int page, int h, int L, int key0, uint32_t dst,
                                        unsigned* err) const {
    const int key = key0 + rbase;
    int left = L - key;  // rows of this thread that exist
    const __nv_bfloat16 *ks = c.k, *vs = c.v;
    if (left > 0) {
      if (page >= 0 && page < c.num_pages) {
        const int64_t off = page * c.page_stride + (key & ((1 << c.page_shift) - 1)) * c.row_stride +
                            h * c.head_stride + col * 8;
        ks += off;
        vs += off;
      } else {
        left = 0;
        atomicOr(err, kErrBadOffsets);
      }
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const uint32_t at = dst + Cfg::at(rbase + i, col);
      const uint32_t bytes = i < left ? 16u : 0u;
      const int64_t step = i < left ? i * c.row_stride : 0;
      ptx::cp_async16(at, ks + step, bytes);
      ptx::cp_async16(at + Cfg::kTileBytes, vs + step, bytes);
    }
  }
};

// The arithmetic of one item in one warp: its query rows, what each of them sees, and O.  R rows at most,
// 16 or 8: the product takes the R rows as its 16 rows, or, transposed (S' = K Q', O' = V' P'), as its
// 8 columns, which halves the products, the SiLU and the registers of a call for up to 8 rows.
//   visible: keys [0, lim) and `self`; U: history length, p0: position of row 0.
template <int D, int R>
struct RowsMath;

// h = alpha s / 2 -> silu(alpha s) = h + h tanh(h); an invisible pair is selected to zero.  Its callers round the
// weight to bf16 (half a step, 2^-8 of it): the product with V takes 16-bit operands, and bf16 keeps the range of
// scores, as in hstu_fwd_kernel.  The fp32 sums that it goes into are rounded once, at the end.
__device__ __forceinline__ float rows_silu(float s, float half_alpha, bool visible) {
  const float h = s * half_alpha;
  const float p = fmaf(h, ptx::tanh_approx(h), h);
  return visible ? p : 0.0f;
}

template <int D>
struct RowsMath<D, 16> {
  using Cfg = RowsCfg<D>;
  static constexpr int kAcc = D / 8;
  uint32_t qf[D / 16][4];  // rows lane / 4 (+ 8), columns 2 (lane % 4) + {0, 1, 8, 9} of each 16
  float o[kAcc][4];        // [j]: rows lane / 4 (+ 8), columns 8 j + 2 (lane % 4) + {0, 1}
  int lim[2], self[2];     // rows lane / 4 and + 8
  int U, p0;

  __device__ __forceinline__ void open(const __nv_bfloat16* q, int64_t q_ld, int nrows, int first_pos, int hist) {
    const int lane = threadIdx.x & 31, g = lane >> 2, c2 = (lane & 3) * 2;
#pragma unroll
    for (int ks = 0; ks < D / 16; ++ks)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int r = g + (e & 1) * 8;
        qf[ks][e] = r < nrows ? *reinterpret_cast<const uint32_t*>(q + r * q_ld + c2 + ks * 16 + (e >> 1) * 8) : 0u;
      }
    U = hist;
    p0 = first_pos;
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      self[e] = p0 + g + e * 8;
      lim[e] = self[e] < U ? self[e] + 1 : U;
    }
#pragma unroll
    for (int j = 0; j < kAcc; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e) o[j][e] = 0.0f;
  }

  // O += P V for this warp's quarter of the tile whose first key is j0 and whose buffer is at `buf`.
  __device__ __forceinline__ void tile(int j0, uint32_t buf, float half_alpha) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int c2 = (lane & 3) * 2;
    const int m = lane >> 3, mr = lane & 7;  // ldmatrix: matrix and row this lane addresses
    const uint32_t sk = buf, sv = buf + Cfg::kTileBytes;
    const bool full = j0 + Cfg::kKeys <= U && j0 + Cfg::kKeys <= p0 + 1;
#pragma unroll
    for (int kb = 0; kb < Cfg::kWarpKeys / 16; ++kb) {
      const int key0 = warp * Cfg::kWarpKeys + kb * 16;  // first of this step's 16 keys in the tile
      float s[2][4] = {};
#pragma unroll
      for (int ks = 0; ks < D / 16; ++ks) {
        uint32_t kf[4];
        ptx::ldmatrix4(kf, sk + Cfg::at(key0 + (m >> 1) * 8 + mr, ks * 2 + (m & 1)));
        ptx::mma_16816(s[0], qf[ks], kf[0], kf[1]);
        ptx::mma_16816(s[1], qf[ks], kf[2], kf[3]);
      }
#pragma unroll
      for (int n = 0; n < 2; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int j = j0 + key0 + n * 8 + c2 + (e & 1);
          s[n][e] = rows_silu(s[n][e], half_alpha, full || j < lim[e >> 1] || j == self[e >> 1]);
        }
      const uint32_t pf[4] = {pack_bf16x2(s[0][0], s[0][1]), pack_bf16x2(s[0][2], s[0][3]),
                              pack_bf16x2(s[1][0], s[1][1]), pack_bf16x2(s[1][2], s[1][3])};
#pragma unroll
      for (int jn = 0; jn < D / 16; ++jn) {
        uint32_t vf[4];
        ptx::ldmatrix4_trans(vf, sv + Cfg::at(key0 + (m & 1) * 8 + mr, jn * 2 + (m >> 1)));
        ptx::mma_16816(o[2 * jn], pf, vf[0], vf[1]);
        ptx::mma_16816(o[2 * jn + 1], pf, vf[2], vf[3]);
      }
    }
  }

  // f(row, column, x, y): two neighbouring columns, twice, of the four values that lane `lane` holds as o[j].
  template <typename F>
  __device__ static __forceinline__ void each(int j, int lane, float4 v, F&& f) {
    const int r = lane >> 2, c = j * 8 + (lane & 3) * 2;
    f(r, c, v.x, v.y);
    f(r + 8, c, v.z, v.w);
  }
};

template <int D>
struct RowsMath<D, 8> {
  using Cfg = RowsCfg<D>;
  static constexpr int kAcc = D / 16;
  uint32_t qf[D / 16][2];  // row lane / 4, columns 2 (lane % 4) + {0, 1} and + 8 of each 16
  float o[kAcc][4];        // [j]: columns 16 j + lane / 4 (+ 8 in the second pair), rows 2 (lane % 4) + {0, 1}
  int lim[2], self[2];     // rows 2 (lane % 4) and + 1
  int U, p0;

  __device__ __forceinline__ void open(const __nv_bfloat16* q, int64_t q_ld, int nrows, int first_pos, int hist) {
    const int lane = threadIdx.x & 31, g = lane >> 2, c2 = (lane & 3) * 2;
#pragma unroll
    for (int ks = 0; ks < D / 16; ++ks)
#pragma unroll
      for (int e = 0; e < 2; ++e)
        qf[ks][e] = g < nrows ? *reinterpret_cast<const uint32_t*>(q + g * q_ld + c2 + ks * 16 + e * 8) : 0u;
    U = hist;
    p0 = first_pos;
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      self[e] = p0 + c2 + e;
      lim[e] = self[e] < U ? self[e] + 1 : U;
    }
#pragma unroll
    for (int j = 0; j < kAcc; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e) o[j][e] = 0.0f;
  }

  __device__ __forceinline__ void tile(int j0, uint32_t buf, float half_alpha) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int g = lane >> 2;
    const int m = lane >> 3, mr = lane & 7;  // ldmatrix: matrix and row this lane addresses
    const uint32_t sk = buf, sv = buf + Cfg::kTileBytes;
    const bool full = j0 + Cfg::kKeys <= U && j0 + Cfg::kKeys <= p0 + 1;
#pragma unroll
    for (int kb = 0; kb < Cfg::kWarpKeys / 16; ++kb) {
      const int key0 = warp * Cfg::kWarpKeys + kb * 16;  // first of this step's 16 keys in the tile
      // S': keys lane / 4 (+ 8), rows 2 (lane % 4) + {0, 1}; two chains of products, added.
      float s[2][4] = {};
#pragma unroll
      for (int ks = 0; ks < D / 16; ++ks) {
        uint32_t kf[4];
        ptx::ldmatrix4(kf, sk + Cfg::at(key0 + (m & 1) * 8 + mr, ks * 2 + (m >> 1)));
        ptx::mma_16816(s[ks & 1], kf, qf[ks][0], qf[ks][1]);
      }
      float p[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int j = j0 + key0 + g + (e >> 1) * 8;
        p[e] = rows_silu(s[0][e] + s[1][e], half_alpha, full || j < lim[e & 1] || j == self[e & 1]);
      }
      // P' as the 16 x 8 operand: keys 2 (lane % 4) + {0, 1} (+ 8), row lane / 4.
      const uint32_t p0f = ptx::transpose_8x8(pack_bf16x2(p[0], p[1]));
      const uint32_t p1f = ptx::transpose_8x8(pack_bf16x2(p[2], p[3]));
#pragma unroll
      for (int jn = 0; jn < D / 16; ++jn) {
        uint32_t vf[4];
        ptx::ldmatrix4_trans(vf, sv + Cfg::at(key0 + (m >> 1) * 8 + mr, jn * 2 + (m & 1)));
        ptx::mma_16816(o[jn], vf, p0f, p1f);
      }
    }
  }

  template <typename F>
  __device__ static __forceinline__ void each(int j, int lane, float4 v, F&& f) {
    const int c = j * 16 + (lane >> 2), r = (lane & 3) * 2;
    f(r, c, v.x);
    f(r + 1, c, v.y);
    f(r, c + 8, v.z);
    f(r + 1, c + 8, v.w);
  }
};

__device__ __forceinline__ void rows_put(float* to, float x) { *to = x; }
__device__ __forceinline__ void rows_put(float* to, float x, float y) {
  *reinterpret_cast<float2*>(to) = make_float2(x, y);
}
__device__ __forceinline__ void rows_put(__nv_bfloat16* to, float x) { *to = __float2bfloat16_rn(x); }
__device__ __forceinline__ void rows_put(__nv_bfloat16* to, float x, float y) {
  *reinterpret_cast<uint32_t*>(to) = pack_bf16x2(x, y);
}

__device__ __forceinline__ float4 add4(float4 a, float4 b) {
  return make_float4(a.x + b.x, a.y + b.y, a.z + b.z, a.w + b.w);
}

// Columns 4 quad .. + 4 of output row `row`, head h.
template <int D>
__device__ __forceinline__ void rows_store(const RowsArgs& p, int row, int h, int quad, float4 a) {
  const uint2 w = make_uint2(pack_bf16x2(a.x * p.inv_n, a.y * p.inv_n), pack_bf16x2(a.z * p.inv_n, a.w * p.inv_n));
  *reinterpret_cast<uint2*>(p.out + (int64_t)row * p.out_ld + (int64_t)h * D + quad * 4) = w;
}

// ---------------------------------------------------------------------------------------------
// One cluster for each item
// ---------------------------------------------------------------------------------------------
template <int D, int R>
__global__ void __launch_bounds__(kRowsThreads, 2) paged_rows_kernel(const RowsArgs p) {
  using Cfg = RowsCfg<D>;
  using Math = RowsMath<D, R>;
  extern __shared__ __align__(128) uint8_t rows_smem[];
  const uint32_t sbase = ptx::smem_addr(rows_smem);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int split = (int)ptx::cluster_ctarank();
  const int S = (int)(gridDim.x / ptx::nclusters_x());
  const int item = (int)ptx::cluster_id_x();
  const int bh = item / p.blocks, blk = item - bh * p.blocks;
  const int b = bh / p.H, h = bh - b * p.H;

  asm volatile("griddepcontrol.wait;" ::: "memory");
  const PagedUser u = paged_user(p.cache, p.q_offsets, p.kv_len, p.num_targets, b, p.total_new, p.max_new, p.max_kv);
  if (split == 0 && h == 0 && blk == 0 && tid == 0) {
    bool bad = !u.ok;
    if (b == 0) bad |= p.q_offsets[0] != 0 || p.q_offsets[p.B] != p.total_new;
    if (bad) atomicOr(p.err, kErrBadOffsets);
  }
  const int r0 = blk * kRowsBlock, nrows = min(kRowsBlock, u.n - r0);
  if (!u.ok || nrows <= 0) return;  // the whole cluster agrees
  const int row0 = u.q0 + r0, pos0 = u.L - u.n + r0;

  // This CTA's share of the visible key tiles.
  const TileRange range = key_tiles<Cfg::kKeys>(pos0, pos0 + nrows, u.L - u.T);
  const int ntiles = tile_count(range);
  const int t_begin = (int)((int64_t)ntiles * split / S), t_end = (int)((int64_t)ntiles * (split + 1) / S);

  const RowsCopy<D> copy;
  auto key_of = [&](int t) { return tile_at(range, t) * Cfg::kKeys; };
  int page = t_begin < t_end ? copy.look_up(p.cache, b, u.L, key_of(t_begin)) : 0;
  auto fetch = [&](int t, int stage) {
    if (t < t_end) {
      const int here = page;
      if (t + 1 < t_end) page = copy.look_up(p.cache, b, u.L, key_of(t + 1));
      copy.issue(p.cache, here, h, u.L, key_of(t), sbase + stage * Cfg::kStageBytes, p.err);
    }
    ptx::cp_async_commit();
  };
#pragma unroll
  for (int s = 0; s < kRowsStages - 1; ++s) fetch(t_begin + s, s);
  Math math;
  math.open(p.q + (int64_t)row0 * p.q_ld + (int64_t)h * D, p.q_ld, nrows, pos0, u.L - u.T);

  int stage = 0;
  for (int t = t_begin; t < t_end; ++t) {
    ptx::cp_async_wait<kRowsStages - 2>();
    __syncthreads();
    fetch(t + kRowsStages - 1, stage == 0 ? kRowsStages - 1 : stage - 1);  // consumed in the previous step
    math.tile(key_of(t), sbase + stage * Cfg::kStageBytes, p.half_alpha);
    stage = stage + 1 == kRowsStages ? 0 : stage + 1;
  }

  // The four warps' sums, then the cluster's.
  ptx::cp_async_wait<0>();
  __syncthreads();
  float* part = reinterpret_cast<float*>(rows_smem);  // [4][R][kPitch]
  constexpr int kPitch = D + (R == 16 ? 8 : 4), kQuads = kPitch / 4;  // a warp's stores hit 32 banks
  float* mine = part + warp * R * kPitch;
#pragma unroll
  for (int j = 0; j < Math::kAcc; ++j)
    Math::each(j, lane, make_float4(math.o[j][0], math.o[j][1], math.o[j][2], math.o[j][3]),
               [&](int r, int c, auto... v) { rows_put(mine + r * kPitch + c, v...); });
  __syncthreads();
  const int quads = nrows * (D / 4);
  for (int i = tid; i < quads; i += kRowsThreads) {
    const int r = i / (D / 4), c = i % (D / 4);
    float4* at = reinterpret_cast<float4*>(part) + r * kQuads + c;
    float4 a = *at;
#pragma unroll
    for (int w = 1; w < 4; ++w) a = add4(a, at[w * R * kQuads]);
    if (S > 1) *at = a;
    else rows_store<D>(p, row0 + r, h, c, a);
  }
  if (S == 1) return;
  ptx::cluster_sync();
  for (int i = split * kRowsThreads + tid; i < quads; i += S * kRowsThreads) {
    const int r = i / (D / 4), c = i % (D / 4);
    float4 a = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 8
    for (int w = 0; w < S; ++w) a = add4(a, ptx::ld_cluster_v4(ptx::mapa_shared(sbase + (r * kQuads + c) * 16, w)));
    rows_store<D>(p, row0 + r, h, c, a);
  }
  ptx::cluster_sync();  // no CTA leaves while its sums are read
}

// ---------------------------------------------------------------------------------------------
// Equal runs of tiles
// ---------------------------------------------------------------------------------------------
constexpr int kRunUsers = 1024;   // users whose first tiles a CTA keeps in shared memory
constexpr int kRunMinTiles = 2;   // a run is at least this long

// Tiles x in [0, tiles) of all items are dealt out in `runs` runs (runs <= tiles: none is empty).
__device__ __forceinline__ int run_begin(int tiles, int runs, int r) { return (int)((int64_t)tiles * r / runs); }
__device__ __forceinline__ int run_of(int tiles, int runs, int x) {
  int r = (int)((int64_t)x * runs / tiles);
  while (r + 1 < runs && run_begin(tiles, runs, r + 1) <= x) ++r;
  while (r > 0 && run_begin(tiles, runs, r) > x) --r;
  return r;
}

struct RunsArgs {
  RowsArgs rows;
  // Item (user b, head h) is b * H + h.  parts[item] = {first run, last run} of its tiles, written by the
  // CTA of its first tile.  An item of one run is written to `out` at once.  Otherwise its first part's
  // sums are in slot 2 * (first run) + 1 and every other run r's in slot 2 * r: [slot][16][D] floats.
  int2* parts;
  float* sums;
};

template <int D, int R>
__global__ void __launch_bounds__(kRowsThreads, 2) paged_rows_run_kernel(const RunsArgs a) {
  using Cfg = RowsCfg<D>;
  using Math = RowsMath<D, R>;
  const RowsArgs& p = a.rows;
  extern __shared__ __align__(128) uint8_t rows_smem[];
  const uint32_t sbase = ptx::smem_addr(rows_smem);
  __shared__ int s_first[kRunUsers + 1];  // first tile of each user
  __shared__ int s_warp[kRowsThreads / 32];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;

  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  // Tiles of every user, scanned: thread t takes users [t * per, (t + 1) * per).
  auto user = [&](int b) {
    return paged_user(p.cache, p.q_offsets, p.kv_len, p.num_targets, b, p.total_new, p.max_new, p.max_kv);
  };
  auto tiles_of = [&](const PagedUser& u) { return key_tiles<Cfg::kKeys>(u.L - u.n, u.L, u.L - u.T); };
  const int per = (p.B + kRowsThreads - 1) / kRowsThreads;
  int mine = 0;
  bool bad = blockIdx.x == 0 && tid == 0 && (p.q_offsets[0] != 0 || p.q_offsets[p.B] != p.total_new);
  for (int b = tid * per; b < min(p.B, (tid + 1) * per); ++b) {
    const PagedUser u = user(b);
    bad |= !u.ok;
    const int n = u.ok && u.n > 0 ? tile_count(tiles_of(u)) * p.H : 0;
    s_first[b] = n;
    mine += n;
  }
  if (bad && blockIdx.x == 0) atomicOr(p.err, kErrBadOffsets);
  int incl = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int n = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += n;
  }
  if (lane == 31) s_warp[warp] = incl;
  __syncthreads();
  int at = incl - mine, tiles = 0;
#pragma unroll
  for (int w = 0; w < kRowsThreads / 32; ++w) {
    if (w < warp) at += s_warp[w];
    tiles += s_warp[w];
  }
  for (int b = tid * per; b < min(p.B, (tid + 1) * per); ++b) {
    const int n = s_first[b];
    s_first[b] = at;
    at += n;
  }
  if (tid == 0) s_first[p.B] = tiles;
  __syncthreads();
  const int most = tiles / kRunMinTiles;
  const int runs = most < 1 ? 1 : min(most, (int)gridDim.x);
  const int run = blockIdx.x;
  if (tiles == 0 || run >= runs) return;
  const int x0 = run_begin(tiles, runs, run), x1 = run_begin(tiles, runs, run + 1);

  // A place in the run: tile t of the n tiles of (b, h).
  struct Cursor {
    int b, h, t, n;
    PagedUser u;
    TileRange range;
  };
  auto enter = [&](Cursor& c, int b) {
    c.b = b;
    c.u = user(b);
    c.range = tiles_of(c.u);
    c.n = tile_count(c.range);
  };
  auto advance = [&](Cursor& c) {
    if (++c.t < c.n) return;
    c.t = 0;
    if (++c.h < p.H) return;
    c.h = 0;
    int b = c.b + 1;
    while (s_first[b + 1] == s_first[b]) ++b;  // users without tiles; the run ends before the users do
    enter(c, b);
  };
  auto key_of = [&](const Cursor& c) { return tile_at(c.range, c.t) * Cfg::kKeys; };
  Cursor eat;
  enter(eat, owner_of(s_first, p.B, x0));
  eat.h = (x0 - s_first[eat.b]) / eat.n;
  eat.t = (x0 - s_first[eat.b]) - eat.h * eat.n;
  Cursor ahead = eat;  // the next tile to fetch; its table entry is in `page`

  const RowsCopy<D> copy;
  int fetched = x0;
  int page = copy.look_up(p.cache, ahead.b, ahead.u.L, key_of(ahead));
  auto fetch = [&](int stage) {
    if (fetched < x1) {
      const int here = page, key0 = key_of(ahead), hh = ahead.h, L = ahead.u.L;
      if (++fetched < x1) {
        advance(ahead);
        page = copy.look_up(p.cache, ahead.b, ahead.u.L, key_of(ahead));
      }
      copy.issue(p.cache, here, hh, L, key0, sbase + stage * Cfg::kStageBytes, p.err);
    }
    ptx::cp_async_commit();
  };
#pragma unroll
  for (int s = 0; s < kRowsStages - 1; ++s) fetch(s);
  Math math;
  bool fresh = true;
  int first_t = 0;  // the item's tile that this CTA began with
  int stage = 0;
  for (int x = x0; x < x1; ++x) {
    if (fresh) {
      math.open(p.q + (int64_t)eat.u.q0 * p.q_ld + (int64_t)eat.h * D, p.q_ld, eat.u.n, eat.u.L - eat.u.n,
                eat.u.L - eat.u.T);
      fresh = false;
      first_t = eat.t;
    }
    ptx::cp_async_wait<kRowsStages - 2>();
    __syncthreads();
    fetch(stage == 0 ? kRowsStages - 1 : stage - 1);
    math.tile(key_of(eat), sbase + stage * Cfg::kStageBytes, p.half_alpha);
    const bool last = eat.t + 1 == eat.n;
    if (last || x + 1 == x1) {
      // The end of the item or of the run: the warps' sums meet in the tile's buffer, which is free until
      // the next step's barrier, as [warp][j][lane] float4; then the threads add the four.
      float4* red = reinterpret_cast<float4*>(rows_smem + stage * Cfg::kStageBytes);
      __syncthreads();
#pragma unroll
      for (int j = 0; j < Math::kAcc; ++j)
        red[(warp * Math::kAcc + j) * 32 + lane] = make_float4(math.o[j][0], math.o[j][1], math.o[j][2], math.o[j][3]);
      __syncthreads();
      const bool head = first_t == 0, whole = head && last;
      float* slot = a.sums + (size_t)(2 * run + (head ? 1 : 0)) * kRowsBlock * D;
      __nv_bfloat16* out = p.out + (int64_t)eat.u.q0 * p.out_ld + (int64_t)eat.h * D;
      for (int i = tid; i < Math::kAcc * 32; i += kRowsThreads) {
        float4 v = red[i];
#pragma unroll
        for (int w = 1; w < 4; ++w) v = add4(v, red[w * Math::kAcc * 32 + i]);
        Math::each(i >> 5, i & 31, v, [&](int r, int c, auto... x) {
          if (r >= eat.u.n) return;
          if (whole) rows_put(out + r * p.out_ld + c, x * p.inv_n...);
          else rows_put(slot + r * D + c, x...);
        });
      }
      if (head && tid == 0)
        a.parts[(int64_t)eat.b * p.H + eat.h] = make_int2(run, run_of(tiles, runs, x + eat.n - 1 - eat.t));
      fresh = true;
    }
    stage = stage + 1 == kRowsStages ? 0 : stage + 1;
    if (x + 1 < x1) advance(eat);
  }
}

// Adds the parts of the items that several runs share: one CTA for each item, groups of threads taking
// every kGroups-th part, then the groups' sums in order.
constexpr int kSumThreads = 256;

template <int D>
__global__ void __launch_bounds__(kSumThreads) paged_rows_sum_kernel(const RunsArgs a) {
  __shared__ float4 s_sum[kSumThreads];
  const RowsArgs& p = a.rows;
  const int b = blockIdx.x / p.H, h = blockIdx.x - b * p.H;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int2 runs = a.parts[blockIdx.x];  // not written for a user without tiles
  const PagedUser u = paged_user(p.cache, p.q_offsets, p.kv_len, p.num_targets, b, p.total_new, p.max_new, p.max_kv);
  if (!u.ok || u.n == 0 || runs.x == runs.y) return;
  const int quads = u.n * (D / 4);
  int lanes = D / 4;  // threads of a group: a power of two, at least a row's quads
  while (lanes < quads && lanes < kSumThreads) lanes *= 2;
  const int groups = kSumThreads / lanes, group = threadIdx.x / lanes;
  const float4* sums = reinterpret_cast<const float4*>(a.sums);
  constexpr int kSlot = kRowsBlock * D / 4;
  for (int i0 = 0; i0 < quads; i0 += lanes) {
    const int i = i0 + threadIdx.x % lanes;
    float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    if (i < quads) {
#pragma unroll 8
      for (int r = runs.x + group; r <= runs.y; r += groups)
        v = add4(v, sums[(size_t)(2 * r + (r == runs.x)) * kSlot + i]);
    }
    if (groups > 1) {
      s_sum[threadIdx.x] = v;
      __syncthreads();
      if (group == 0)
        for (int k = 1; k < groups; ++k) v = add4(v, s_sum[k * lanes + threadIdx.x]);
    }
    if (group == 0 && i < quads) rows_store<D>(p, u.q0 + i / (D / 4), h, i % (D / 4), v);
  }
}

}  // namespace hstu
