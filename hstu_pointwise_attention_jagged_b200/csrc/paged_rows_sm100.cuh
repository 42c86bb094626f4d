// paged_rows_sm100.cuh — target-aware SiLU attention of a few new rows a user over the paged cache.
//
// With up to 16 query rows a user the work is a pass over the user's cached K and V: 2 * L * d * 2
// bytes a head for at most 16 * L * d * 4 flops, so the bound is DRAM and the tensor cores only have
// to stay out of the way.  A 128-row tcgen05 tile would be empty but for those rows; the warp-level
// m16n8k16 product takes exactly 16 rows from shared memory and keeps S, P and O in registers.
//
// One cluster of S CTAs serves one (user, head, block of 16 rows): SiLU attention has no softmax
// statistics, so the key tiles are shared out in S runs and the partial O's simply add up, over
// distributed shared memory, in rank order (the sum does not depend on timing).  No workspace, no
// second launch.  Each CTA streams its run through kStages tiles of cp.async copies; the four warps
// take a quarter of each tile's keys, each with its own O, summed at the end.
//
// A tile is 16 KB of K and 16 KB of V: 64, 128 or 256 keys for d = 128, 64, 32, so that every thread
// copies 8 consecutive rows of one 16-byte column; 8 aligned rows never cross a page.  Rows past
// the user's length are filled with zeros, whatever the page holds there.
#pragma once

#include <climits>
#include <cstdint>
#include <cuda_bf16.h>

#include "hstu_fwd_sm100.cuh"
#include "paged_cache.cuh"
#include "schedule.cuh"
#include "sm100_ptx.cuh"

namespace hstu {

constexpr int kRowsThreads = 128;
constexpr int kRowsBlock = 16;     // query rows of a cluster
constexpr int kRowsStages = 3;
constexpr int kRowsMaxSplit = 16;  // CTAs of a cluster

template <int D>
struct RowsCfg {
  static constexpr int kRowBytes = D * 2;
  static constexpr int kChunks = kRowBytes / 16;     // 16-byte columns of a row
  static constexpr int kKeys = 64 * 128 / D;         // keys of a tile
  static constexpr int kWarpKeys = kKeys / 4;
  static constexpr int kTileBytes = kKeys * kRowBytes;  // 16 KB
  static constexpr int kSmemBytes = kRowsStages * 2 * kTileBytes;
  static_assert(4 * kRowsBlock * D * 4 <= kSmemBytes, "the warps' partial sums reuse the tiles");
  // Physical column of logical column c in row r: eight consecutive rows hit eight 16-byte bank groups.
  __device__ static __forceinline__ int column(int r, int c) {
    return D == 32 ? (c ^ ((r >> 1) & 3)) : (c ^ (r & 7));
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
  int32_t B, H, blocks, total_new, max_new, max_kv;  // blocks: 16-row blocks of a user (upper bound)
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

template <int D>
__global__ void __launch_bounds__(kRowsThreads, 2) paged_rows_kernel(const RowsArgs p) {
  using Cfg = RowsCfg<D>;
  extern __shared__ __align__(128) uint8_t rows_smem[];
  const uint32_t sbase = ptx::smem_addr(rows_smem);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int split = (int)ptx::cluster_ctarank();
  // Cluster index -> user, head, block of rows.
  const int S = (int)(gridDim.x / ptx::nclusters_x());
  int x = (int)ptx::cluster_id_x();
  const int blk = x % p.blocks;
  x /= p.blocks;
  const int h = x % p.H, b = x / p.H;

  asm volatile("griddepcontrol.wait;" ::: "memory");
  const PagedUser u = paged_user(p.cache, p.q_offsets, p.kv_len, p.num_targets, b, p.total_new, p.max_new, p.max_kv);
  if (split == 0 && h == 0 && blk == 0 && tid == 0) {
    bool bad = !u.ok;
    if (b == 0) bad |= p.q_offsets[0] != 0 || p.q_offsets[p.B] != p.total_new;
    if (bad) atomicOr(p.err, kErrBadOffsets);
  }
  const int r0 = blk * kRowsBlock;
  // The whole cluster agrees: nothing to do.
  if (!u.ok || r0 >= u.n) return;
  const int nrows = min(kRowsBlock, u.n - r0);
  const int U = u.L - u.T;
  const int p0 = u.L - u.n + r0;  // position of the first row

  // This CTA's run of the visible key tiles.
  const TileRange range = key_tiles<Cfg::kKeys>(p0, p0 + nrows, U);
  const int ntiles = tile_count(range);
  const int t_begin = (int)((int64_t)ntiles * split / S), t_end = (int)((int64_t)ntiles * (split + 1) / S);

  // Copies: thread -> 16-byte column tid % kChunks of rows 8 (tid / kChunks) .. + 8.
  const int col = tid % Cfg::kChunks, rbase = (tid / Cfg::kChunks) * 8;
  const int32_t* table = p.cache.table + b * p.cache.table_ld;
  const int64_t head_off = h * p.cache.head_stride + col * 8;
  const int page_mask = (1 << p.cache.page_shift) - 1;
  auto issue = [&](int t, int stage) {
    const int key = tile_at(range, t) * Cfg::kKeys + rbase;
    int left = u.L - key;  // rows of this thread that exist
    const __nv_bfloat16 *ks = p.cache.k, *vs = p.cache.v;
    if (left > 0) {
      const int page = table[key >> p.cache.page_shift];
      if (page >= 0 && page < p.cache.num_pages) {
        const int64_t off = page * p.cache.page_stride + (key & page_mask) * p.cache.row_stride + head_off;
        ks += off;
        vs += off;
      } else {
        left = 0;
        atomicOr(p.err, kErrBadOffsets);
      }
    }
    const uint32_t dk = sbase + stage * 2 * Cfg::kTileBytes;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int r = rbase + i;
      const uint32_t at = r * Cfg::kRowBytes + Cfg::column(r, col) * 16;
      const uint32_t bytes = i < left ? 16u : 0u;
      const int64_t step = i < left ? i * p.cache.row_stride : 0;
      ptx::cp_async16(dk + at, ks + step, bytes);
      ptx::cp_async16(dk + Cfg::kTileBytes + at, vs + step, bytes);
    }
  };
#pragma unroll
  for (int s = 0; s < kRowsStages - 1; ++s) {
    if (t_begin + s < t_end) issue(t_begin + s, s);
    ptx::cp_async_commit();
  }

  // Q as the A operand: rows lane / 4 and + 8, columns 2 (lane % 4) + {0, 1, 8, 9} of each 16.
  const int g = lane >> 2, c2 = (lane & 3) * 2;
  uint32_t qf[D / 16][4];
  {
    const __nv_bfloat16* q = p.q + (int64_t)(u.q0 + r0) * p.q_ld + (int64_t)h * D + c2;
#pragma unroll
    for (int ks = 0; ks < D / 16; ++ks) {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int r = g + (e & 1) * 8;
        qf[ks][e] = r < nrows ? *reinterpret_cast<const uint32_t*>(q + r * p.q_ld + ks * 16 + (e >> 1) * 8) : 0u;
      }
    }
  }
  // Row lane / 4 (+ 8): keys [0, lim) and `self` are visible.
  int lim[2], self[2];
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    self[e] = p0 + g + e * 8;
    lim[e] = self[e] < U ? self[e] + 1 : U;
  }

  float o[D / 8][4];
#pragma unroll
  for (int j = 0; j < D / 8; ++j)
#pragma unroll
    for (int e = 0; e < 4; ++e) o[j][e] = 0.0f;

  const int m = lane >> 3, mr = lane & 7;  // ldmatrix: matrix and row this lane addresses
  int stage = 0;
  for (int t = t_begin; t < t_end; ++t) {
    ptx::cp_async_wait<kRowsStages - 2>();
    __syncthreads();
    {
      const int next = t + kRowsStages - 1;
      const int into = stage == 0 ? kRowsStages - 1 : stage - 1;  // consumed in the previous step
      if (next < t_end) issue(next, into);
      ptx::cp_async_commit();
    }
    const uint32_t sk = sbase + stage * 2 * Cfg::kTileBytes, sv = sk + Cfg::kTileBytes;
    const int j0 = tile_at(range, t) * Cfg::kKeys;
    const bool full = j0 + Cfg::kKeys <= U && j0 + Cfg::kKeys <= p0 + 1;
#pragma unroll
    for (int kb = 0; kb < Cfg::kWarpKeys / 16; ++kb) {
      const int key0 = warp * Cfg::kWarpKeys + kb * 16;  // first of this step's 16 keys in the tile
      float s[2][4] = {};
#pragma unroll
      for (int ks = 0; ks < D / 16; ++ks) {
        uint32_t kf[4];
        const int r = key0 + (m >> 1) * 8 + mr;
        ptx::ldmatrix4(kf, sk + r * Cfg::kRowBytes + Cfg::column(r, ks * 2 + (m & 1)) * 16);
        ptx::mma_16816(s[0], qf[ks], kf[0], kf[1]);
        ptx::mma_16816(s[1], qf[ks], kf[2], kf[3]);
      }
      // p = silu(alpha s) = hx + hx tanh(hx), hx = alpha s / 2; masked pairs select zero.
#pragma unroll
      for (int n = 0; n < 2; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float hx = s[n][e] * p.half_alpha;
          float v = fmaf(hx, ptx::tanh_approx(hx), hx);
          if (!full) {
            const int j = j0 + key0 + n * 8 + c2 + (e & 1);
            v = (j < lim[e >> 1] || j == self[e >> 1]) ? v : 0.0f;
          }
          s[n][e] = v;
        }
      const uint32_t pf[4] = {pack_bf16x2(s[0][0], s[0][1]), pack_bf16x2(s[0][2], s[0][3]),
                              pack_bf16x2(s[1][0], s[1][1]), pack_bf16x2(s[1][2], s[1][3])};
#pragma unroll
      for (int jn = 0; jn < D / 16; ++jn) {
        uint32_t vf[4];
        const int r = key0 + (m & 1) * 8 + mr;
        ptx::ldmatrix4_trans(vf, sv + r * Cfg::kRowBytes + Cfg::column(r, jn * 2 + (m >> 1)) * 16);
        ptx::mma_16816(o[2 * jn], pf, vf[0], vf[1]);
        ptx::mma_16816(o[2 * jn + 1], pf, vf[2], vf[3]);
      }
    }
    stage = stage + 1 == kRowsStages ? 0 : stage + 1;
  }

  // The four warps' sums, then the cluster's.
  ptx::cp_async_wait<0>();
  __syncthreads();
  float* part = reinterpret_cast<float*>(rows_smem);  // [4][16][D]
#pragma unroll
  for (int j = 0; j < D / 8; ++j) {
    float* at = part + (warp * kRowsBlock + g) * D + j * 8 + c2;
    *reinterpret_cast<float2*>(at) = make_float2(o[j][0], o[j][1]);
    *reinterpret_cast<float2*>(at + 8 * D) = make_float2(o[j][2], o[j][3]);
  }
  __syncthreads();
  const int quads = nrows * (D / 4);
  for (int i = tid; i < quads; i += kRowsThreads) {
    float4 a = reinterpret_cast<float4*>(part)[i];
#pragma unroll
    for (int w = 1; w < 4; ++w) {
      const float4 v = reinterpret_cast<float4*>(part + w * kRowsBlock * D)[i];
      a.x += v.x;
      a.y += v.y;
      a.z += v.z;
      a.w += v.w;
    }
    reinterpret_cast<float4*>(part)[i] = a;
  }
  if (S > 1) ptx::cluster_sync(); else __syncthreads();
  for (int i = split * kRowsThreads + tid; i < quads; i += S * kRowsThreads) {
    float4 a = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    if (S == 1) {
      a = reinterpret_cast<float4*>(part)[i];
    } else {
#pragma unroll 8
      for (int w = 0; w < S; ++w) {
        const float4 v = ptx::ld_cluster_v4(ptx::mapa_shared(sbase + i * 16, w));
        a.x += v.x;
        a.y += v.y;
        a.z += v.z;
        a.w += v.w;
      }
    }
    const int r = i / (D / 4), c = (i - r * (D / 4)) * 4;
    const uint2 w = make_uint2(pack_bf16x2(a.x * p.inv_n, a.y * p.inv_n), pack_bf16x2(a.z * p.inv_n, a.w * p.inv_n));
    *reinterpret_cast<uint2*>(p.out + (int64_t)(u.q0 + r0 + r) * p.out_ld + (int64_t)h * D + c) = w;
  }
  if (S > 1) ptx::cluster_sync();  // no CTA leaves while its sums are read
}

}  // namespace hstu
